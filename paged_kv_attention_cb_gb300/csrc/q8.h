// The 8-bit paged cache: launchers and arguments shared by its kernels and the planner.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "merge.h"

namespace cb {

// k, v: [num_blocks, block_size, Hkv, D] e4m3; k_scale, v_scale: [num_blocks, block_size, Hkv]
// e8m0 (one power of two per row).
struct Q8Cache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
};

cudaError_t launch_write_kv_q8(const void* k_new, const void* v_new, const Q8Cache& c,
                               const int64_t* slot_mapping, int32_t num_tokens, int64_t num_slots,
                               int32_t Hkv, int32_t D, int32_t dtype, int32_t* error_word,
                               cudaStream_t stream);

cudaError_t launch_read_kv_q8(void* k_out, void* v_out, const Q8Cache& c,
                              const int64_t* slot_mapping, int32_t num_tokens, int64_t num_slots,
                              int32_t Hkv, int32_t D, int32_t dtype, int32_t* error_word,
                              cudaStream_t stream);

// ---- split kernel (attn_q8.cu): rows of requests with 1 <= q_len <= max_q

constexpr int kQ8KeyBlock = 16;      // keys per unit of work (and per stage of the ring)
constexpr int kQ8MaxStages = 32;
constexpr int kQ8MaxHeads = 8;       // KV heads per CTA
constexpr int kQ8Producers = 4;      // producer warps per CTA (a power of two)
constexpr int kQ8MaxColumnWarps = 4; // warps of a head on different columns
constexpr int kQ8TableCtas = 192;    // CTAs per group of heads (their starts are arguments)
constexpr int kQ8SmemLimit = 232448; // 227 KiB dynamic shared memory per CTA
// Bytes of the ring: a little over the latency times the rate of one SM's share of HBM. More
// only takes L1 away from the query rows and the few spilled registers (16 requests x 32768: 168
// us with 132 KB of stages, 177 with 198 KB, 211 with 66 KB).
constexpr int kQ8RingBytes = 136 * 1024;
// Key blocks a CTA has at least: small steps are latency, and a block of its own for every CTA is
// their shortest way (4 requests of up to 300 positions: 6.7 us, 7.6 from two on).
constexpr int kQ8MinBlocksPerCta = 1;

// Where a CTA's range of key blocks starts (the entry behind the last CTA: the end of all).
struct Q8CtaStart {
  int u;     // global index of the CTA's first key block
  int r;     // its request
  int tile;  // its token tile within the request
  int item;  // index of that (request, tile) among the step's
  int u0;    // global index of the item's first key block
  int t0, q_len, seq;  // the request's first query row, query tokens and KV length
};

struct Q8Args {
  StepArgs a;  // k_cache / v_cache unused
  Q8Cache c;
  int num_ctas;       // CTA b takes the key blocks from start[b].u to start[b + 1].u
  int heads_per_cta;  // HB
  int key_warps;      // KW: warps per KV head and columns; block i goes to those with i % KW
  int column_warps;   // CW: warps per KV head and block, each with 8 NB of the item's columns
  int group_blocks;   // GB: blocks that a producer's lanes issue together (a power of two); block
                      // i belongs to producer i / GB % kQ8Producers
  int stages;         // multiple of KW and of GB * kQ8Producers
  int tile_tokens;    // TT: query tokens per item (TT * G columns, at most 8 NB CW)
  int lg_block;       // log2 of block_size
  int lg_group;       // log2 of query heads per KV head
  int max_q;
  // Steps of decode rows only: the warp that reads a request's last key block quantises the
  // request's new row of its head into the cache and into its staged copy of the block, so the
  // step needs no launch of its own for the write. nullptr: the rows are in the cache already.
  const void* k_new;  // [T, Hkv, D]
  const void* v_new;
  const int64_t* slot_mapping;
  float* part_o;      // [((item + CTA) * KW + key warp) * TT + token][Hq][D]
  float2* part_ml;    // the same rows x [Hq]
  Q8CtaStart start[kQ8TableCtas + 1];
};

// Column blocks (of 8 columns) per warp: 1 or 2.
cudaError_t launch_q8_split(const Q8Args& p, int column_blocks, cudaStream_t stream);
size_t q8_smem_bytes(int D, int HB, int warps, int NB, bool f32, int stages, int Hkv);

// One warp per (row, KV head) on the CUDA cores: every shape, no split.
cudaError_t launch_q8_portable(const StepArgs& a, const Q8Cache& c, cudaStream_t stream);

// ---- whole requests as bf16 pages (kv_q8.cu), for the prefill tiles

constexpr int kDequantMaxEntries = 128;

// Logical pages first .. first + n - 1 of request r become destination pages dst .. dst + n - 1,
// and table[row + first + i] = dst + i. Positions before first_pos are read as zeros.
struct DequantEntry {
  int r, first, n, dst, row, first_pos;
};

struct DequantArgs {
  Q8Cache c;
  const int32_t* block_table;
  int bt_stride;
  int num_blocks, block_size, num_kv_heads, head_dim;
  void *k, *v;     // [pages, block_size, Hkv, D] bf16
  int32_t* table;  // logical page -> destination page, the requests' rows one after the other
  int32_t* error_word;
  int dst0, n_pages;  // destination pages dst0 .. dst0 + n_pages - 1, in the entries' order
  int n_entries;
  DequantEntry entries[kDequantMaxEntries];
};

cudaError_t launch_dequant_pages_q8(const DequantArgs& d, cudaStream_t stream);

}  // namespace cb
