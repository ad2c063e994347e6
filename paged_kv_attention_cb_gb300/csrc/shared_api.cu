// cb_paged_attention_shared (declared in include/cb.h): decode rows of groups of requests whose
// leading pages are the same. With P the prefix of request r's group,
//     out = sum_{p < P} 2^s_p v_p + sum_{P <= p} 2^s_p v_p, over the sum of the weights:
// the first part for all rows of a group at once, as dense tiles of 128 rows on the tensor cores
// that read the prefix's K/V once per 256 rows (prefill_tile_kernel's kSharedPrefix), the second
// row by row from each request's own pages (decode_split_kernel from position P on), joined by
// log-sum-exp (merge.h).
//
// What bounds it: the suffixes are a decode stream (HBM), the prefix is a matrix product of
// rows x P (tensor pipe, 4 Hq D P FLOP a row). The two run side by side: the decode grid leaves
// k SMs to the prefix grid, whose persistent CTAs take the other SMs over as they come free.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "api.h"
#include "cb.h"
#include "launch.h"
#include "merge.h"
#include "plan.h"

namespace {

using cb::report_error;

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kMaxDecodeCtasShared = 192;    // decode CTAs (at most one per SM)
constexpr int kMaxPrefixUnits = 4 * 192;     // units beyond one per (pair of tiles, KV head)

// (row, head) entries of partial results: the decode pieces, and the prefix's.
size_t partial_entries(int64_t R, int64_t T, int64_t Hq) {
  return (size_t)(Hq * (R + kMaxDecodeCtasShared + 2 * T)) + (size_t)256 * kMaxPrefixUnits;
}

size_t shared_bytes(int64_t R, int64_t T, int64_t Hq, int64_t D) {
  const size_t n = partial_entries(R, T, Hq);
  return cb::kWorkspaceHeaderBytes + cb::kWorkspaceAlign + align256(n * 8) + n * D * 4;
}

// Measured on GB300 (32 and 16 rows of 64 query heads behind 131072 positions of 8 KV heads: 106.4
// and 95.5 us): microseconds of one SM for a 128-key tile against two query tiles (tensor pipe and
// softmax) and, in a tail, against one (the keys' bytes: 5.6 TB/s over all SMs); and for a unit's
// start and its partial rows. A tail taken by both softmax groups with one half of each key tile was
// slower than by one of them: 99.0 us there, and with a pair beside it (37 rows in each of four
// groups, 32768 positions) 246 instead of 209 us.
constexpr double kPairUs = 1.9, kTailUs = 1.7, kUnitUs = 4.0;
constexpr double kHbm = 6.6e12;

// The plain step, which reads the shared pages from L2 after the first request: a start of 9 us
// and 0.82 us a key block of its decode partition (64 requests behind 8192 positions, 32/8 heads:
// 187 us; 16 behind 512: 12.6 us). The shared form's launches and merge on top of its model: 9.5 us
// (16 requests behind 2048 positions: 14.7 us shared, 20.7 plain; behind 512: 14.2 and 12.6).
constexpr double kPlainUs = 9.0, kPlainBlockUs = 0.82, kSharedUs = 9.5;

// A decode row's share of the decode grid's time besides its key blocks: its query, first maximum
// and partial rows (148 rows of up to 700 own positions on 12 SMs: 256 us, on 40: 87 us).
constexpr double kDecodeRowUs = 3.0;

struct Group {
  int r, q_start, rows, prefix;
};

struct SharedPlan {
  cb::Plan plan;
  cb::PrefixArgs prefix;
  std::vector<Group> groups;
  std::vector<cb::MergeRow> merge;
  std::vector<int> group_of;  // decode row's group by request, -1: none
  int max_pieces;
};

int rows_per_tile(const cb::StepArgs& a) { return 128 / (a.num_q_heads / a.num_kv_heads); }

// A group's query tiles: pairs of them, and a last one without a second (tail) or not.
struct Tiles {
  int pairs, tail;
};

Tiles tiles_of(const Group& g, const cb::StepArgs& a) {
  const int tq = rows_per_tile(a), tiles = (g.rows + tq - 1) / tq;
  return Tiles{tiles / 2, tiles % 2};
}

int64_t partial_rows(const Group& g, int per) { return (int64_t)cb::prefix_splits(g.prefix, per) * g.rows; }

void plan_prefix(SharedPlan& sp, const cb::StepArgs& a, int per, int grid_max, int first_row) {
  cb::PrefixArgs& p = sp.prefix;
  static_cast<cb::PrefillArgs&>(p) = cb::PrefillArgs{};
  p.a = a;
  p.a.kv_start = nullptr;
  p.tile_tokens = rows_per_tile(a);
  p.box_keys = std::min(a.block_size, 128);
  p.metadata_ready = 1;
  int* header = static_cast<int*>(sp.plan.workspace);
  p.exit_counter = header + cb::kExitCounterOffset / 4;
  p.unit_counter = header + cb::kUnitCounterOffset / 4;
  p.scatter_counter = header + cb::kScatterCounterOffset / 4;
  p.tiles_per_unit = per;
  int row = first_row;
  for (const Group& g : sp.groups) {
    const Tiles t = tiles_of(g, a);
    const int e = p.n_entries++, splits = cb::prefix_splits(g.prefix, per);
    p.entries[e] = cb::PrefillEntry{g.r, 2 * t.pairs + t.tail, g.q_start, g.rows, g.prefix};
    p.part_row[e] = row;
    p.splits[e] = splits;
    p.total_units += (t.pairs + t.tail) * a.num_kv_heads * splits;
    row += (int)partial_rows(g, per);
  }
  p.total_ctas = p.total_units;
  p.grid = std::min(p.total_units, grid_max);
}

// When `units` pieces of work of `us` each are done by k SMs from the start and `rest` more from
// `from` on.
double done_at(long long units, double us, int k, int rest, double from) {
  auto done = [&](double t) {
    return k * (long long)(t / us) + (t > from ? rest * (long long)((t - from) / us) : 0);
  };
  constexpr double kEps = 1e-6;
  double t = ((double)units * us + (rest > 0 ? rest * from : 0.0)) / (k + rest);  // no sooner
  if (t < from) t = (double)units * us / k;
  for (int i = 0; i < 8 && done(t + kEps) < units; ++i) {
    // the next time at which an SM of either kind finishes a piece
    const double a = (floor(t / us + kEps) + 1) * us;
    const double b = t < from ? from + us : from + (floor((t - from) / us + kEps) + 1) * us;
    t = rest > 0 ? std::min(a, b) : a;
  }
  return t;
}

struct Choice {
  int k;      // SMs the decode grid leaves to the prefix grid
  int per;    // key tiles per unit
  double us;  // modelled time
};

// The SM share and the split of the key tiles with the least modelled time: the decode stream on
// its SMs, the prefix's units on the others and then on all, and the merge of the partial rows
// (written and read once at L2's rate).
// decode_us: the decode's time on one SM.
Choice choose(const SharedPlan& sp, const cb::StepArgs& a, double decode_bytes, double decode_us,
              int S, bool beside, size_t max_rows) {
  int longest = 0;
  double tile_us = 0.0;  // of all key tiles
  long long tile_units = 0;
  for (const Group& g : sp.groups) {
    const Tiles t = tiles_of(g, a);
    const int n = cb::prefix_key_tiles(g.prefix);
    tile_us += (double)n * a.num_kv_heads * (t.pairs * kPairUs + t.tail * kTailUs);
    tile_units += (long long)n * a.num_kv_heads * (t.pairs + t.tail);
    longest = std::max(longest, n);
  }
  const double mean_us = tile_us / (double)tile_units;
  const double row_us = (double)a.num_q_heads * a.head_dim * 8 / 4e6;  // a partial row, both ways, on all SMs
  Choice best{4, longest, 1e30};
  // key tiles a unit: 1, 2, 3, 4, 6, 8, 12, 16, ..., and what makes 1 to 4 units per SM
  int candidates[80], n_candidates = 0;
  for (int waves = 1; waves <= 4; ++waves)
    candidates[n_candidates++] = (int)((tile_units + (long long)waves * S - 1) / ((long long)waves * S));
  for (int p2 = 1; p2 < longest; p2 *= 2) {
    candidates[n_candidates++] = p2;
    candidates[n_candidates++] = p2 + p2 / 2;
  }
  candidates[n_candidates++] = longest;
  for (int c = 0; c < n_candidates; ++c) {
    const int per = std::min(candidates[c], longest);
    if (std::find(candidates, candidates + c, per) != candidates + c) continue;
    long long units = 0, rows = 0;
    for (const Group& g : sp.groups) {
      const Tiles t = tiles_of(g, a);
      units += (long long)(t.pairs + t.tail) * a.num_kv_heads * cb::prefix_splits(g.prefix, per);
      rows += partial_rows(g, per);
    }
    if ((size_t)rows <= max_rows) {
      const double us = per * mean_us + kUnitUs;
      for (int k = 4; k < S; k += k < 28 ? 8 : 14) {
        const double td = std::max(decode_bytes / kHbm * 1e6, decode_us / (beside ? S - k : S));
        const double merge = (double)rows * row_us;
        if (std::max(td, (double)units * us / S) + merge >= best.us * 0.97) continue;  // cannot be better
        const double tp = beside ? done_at(units, us, k, S - k, td) : td + done_at(units, us, S, 0, 0.0);
        const double t = std::max(td, tp) + merge;
        if (t < best.us * 0.97) best = Choice{k, per, t};  // (few SMs for the prefix where it makes no odds)
        if (!beside) break;
      }
    }
  }
  return best;
}

// False: the step is better run plainly, or needs a kernel the shared form does not cover.
bool plan_shared(SharedPlan& sp, const cb::StepArgs& a, const int32_t* qsl, const int32_t* seq,
                 const int32_t* prefix, const int32_t* group_start, int n_groups, uint32_t flags,
                 const cb::ScatterInputs* scatter, void* workspace, size_t workspace_bytes) {
  if (a.dtype != CB_BF16 || a.sliding_window > 0 || (flags & CB_FLAG_PORTABLE_ONLY)) return false;
  sp.groups.clear();
  sp.merge.clear();
  sp.group_of.assign(a.num_requests, -1);
  sp.max_pieces = 0;
  for (int g = 0; g < n_groups; ++g) {
    Group gr{-1, 0, 0, 0};
    for (int r = group_start[g]; r < group_start[g + 1]; ++r) {
      if (qsl[r + 1] - qsl[r] != 1 || prefix[r] == 0) continue;
      if (gr.r < 0) gr = Group{r, qsl[r], 0, prefix[r]};
      ++gr.rows;
      sp.group_of[r] = (int)sp.groups.size();
    }
    if (gr.rows == 0) continue;
    sp.groups.push_back(gr);
  }
  if (sp.groups.empty() || sp.groups.size() > cb::kPrefillMaxEntries) return false;

  cb::Plan& plan = sp.plan;
  cb::plan_step(plan, a, qsl, seq, flags, nullptr, workspace, workspace_bytes);
  const int G = a.num_q_heads / a.num_kv_heads;
  if (!plan.fast_decode || plan.portable_mode != -1 || a.block_size % 8 != 0 ||
      !(128 % a.block_size == 0 || a.block_size % 128 == 0) || 128 % G != 0)
    return false;
  plan.concurrent = plan.n_prefill_launches == 0;
  plan.fused_scatter = scatter != nullptr && plan.concurrent;

  long long U = 0, U_plain = 0, decode_rows = 0;
  for (int r = 0; r < a.num_requests; ++r) {
    if (qsl[r + 1] - qsl[r] != 1) continue;
    U += cb::decode_units_host(seq[r], 0, prefix[r]);
    U_plain += cb::decode_units_host(seq[r], 0, 0);
    ++decode_rows;
  }
  const int S = std::min(cb::sm_count(), kMaxDecodeCtasShared);
  const int hg = a.num_kv_heads / plan.decode.heads_per_cta;
  const size_t entries = partial_entries(a.num_requests, a.num_tokens, a.num_q_heads);
  const size_t slots_max = (size_t)a.num_requests + S;
  const double bytes = (double)U * 16 * 2 * a.num_kv_heads * a.head_dim * 2;
  const Choice ch = choose(sp, a, bytes, hg * (U * kPlainBlockUs + decode_rows * kDecodeRowUs), S, plan.concurrent,
                           entries / a.num_q_heads - slots_max);
  const int per = ch.per;
  const double plain_us = kPlainUs + kPlainBlockUs * (double)U_plain * hg / S;
  if (ch.us + kSharedUs >= plain_us && !(flags & CB_FLAG_SHARE_ALWAYS)) return false;
  // (a decode grid larger than its SMs would hold the prefix grid back until its last CTAs start)
  const int C = std::max(1, (plan.concurrent ? S - ch.k : S) / hg);
  const long long slots = a.num_requests + C;
  size_t rows = 0;
  for (const Group& g : sp.groups) rows += (size_t)partial_rows(g, per);
  if ((slots + rows) * a.num_q_heads > entries) return false;
  cb::plan_decode(plan, a, qsl, seq, prefix, U, C, scatter);
  uint8_t* ws = cb::align_workspace(workspace);
  plan.decode.part_ml = reinterpret_cast<float2*>(ws + cb::kWorkspaceHeaderBytes);
  plan.decode.part_o = reinterpret_cast<float*>(ws + cb::kWorkspaceHeaderBytes + align256(entries * 8));
  plan_prefix(sp, a, per, S, (int)slots);
  sp.prefix.concurrent = plan.concurrent ? 1 : 0;
  sp.prefix.part_ml = plan.decode.part_ml;
  sp.prefix.part_o = plan.decode.part_o;

  // ---- the rows in pieces: (request, CTA) slots r + b of the decode, token + split of the prefix
  long long u = 0;
  const int Cn = plan.decode.num_ctas;
  for (int r = 0; r < a.num_requests; ++r) {
    if (qsl[r + 1] - qsl[r] != 1) continue;
    const int n = cb::decode_units_host(seq[r], 0, prefix[r]);
    const int b0 = cb::cta_of_host(u, U, Cn), b1 = cb::cta_of_host(u + n - 1, U, Cn);
    u += n;
    cb::MergeRow m{qsl[r], r + b0, 1, b1 - b0 + 1, 0, 0, 0};
    if (sp.group_of[r] >= 0) {
      const Group& g = sp.groups[sp.group_of[r]];
      m.b = sp.prefix.part_row[sp.group_of[r]] + qsl[r] - g.q_start;
      m.b_step = g.rows;
      m.nb = cb::prefix_splits(g.prefix, per);
    } else if (b1 == b0) {
      continue;
    }
    sp.merge.push_back(m);
    sp.max_pieces = std::max(sp.max_pieces, m.na + m.nb);
  }
  return true;
}

cudaError_t run_shared(SharedPlan& sp, const cb::StepArgs& a, const cb::ScatterInputs* scatter,
                       cudaStream_t s) {
  const cb::Plan& plan = sp.plan;
  cudaError_t e = cudaSuccess;
  if (scatter != nullptr && !plan.fused_scatter)
    e = cb::launch_write_kv(scatter->k_new, scatter->v_new, a.k_cache, a.v_cache, scatter->slot_mapping,
                            a.num_tokens, (int64_t)a.num_blocks * a.block_size,
                            a.num_kv_heads * a.head_dim * 2, a.error_word, s);
  if (e == cudaSuccess) e = cb::launch_decode(plan.decode, plan.decode_plan, s);
  if (e == cudaSuccess) e = cb::launch_prefix(sp.prefix, s);
  for (int l = 0; l < plan.n_prefill_launches && e == cudaSuccess; ++l)
    e = cb::launch_prefill(plan.prefill[l], s);
  if (e != cudaSuccess) return e;
  cb::MergeArgs m;
  m.out = a.out;
  m.dtype = a.dtype;
  m.num_q_heads = a.num_q_heads;
  m.head_dim = a.head_dim;
  m.part_o = plan.decode.part_o;
  m.part_ml = plan.decode.part_ml;
  m.parts = cb::merge_parts(sp.max_pieces);
  return cb::launch_merge(m, sp.merge.data(), (int)sp.merge.size(), s);
}

cb_status attention_shared(void* out, const void* q, void* k_cache, void* v_cache, const void* k_new,
                           const void* v_new, const int64_t* slot_mapping,
                           const int32_t* query_start_loc, const int32_t* seq_lens,
                           const int32_t* block_table, int32_t block_table_stride,
                           const int32_t* prefix_lens, const int32_t* h_query_start_loc,
                           const int32_t* h_seq_lens, const int32_t* h_prefix_lens,
                           const int32_t* h_group_start, int32_t num_groups, int32_t num_requests,
                           int32_t num_tokens, int32_t num_blocks, int32_t block_size,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                           int32_t sliding_window, int32_t dtype, uint32_t flags, void* workspace,
                           size_t workspace_bytes, void* stream) {
  cb_status st = cb::check_step_sizes(num_requests, num_tokens, num_blocks, block_size, num_q_heads,
                                      num_kv_heads, head_dim, block_table_stride, dtype,
                                      h_query_start_loc, h_seq_lens);
  if (st != CB_OK) return st;
  if (num_groups < 0 || (num_groups > 0 && (!h_group_start || !h_prefix_lens)))
    return report_error(CB_ERR_INVALID_ARG, "host mirrors of the groups and prefix_lens are required");
  if (!workspace || workspace_bytes < cb_workspace_size_shared(num_requests, num_tokens, num_q_heads,
                                                               num_kv_heads, head_dim))
    return report_error(CB_ERR_WORKSPACE, "workspace missing or smaller than cb_workspace_size_shared()");
  int64_t max_pages = 0;
  st = cb::check_step_mirrors(h_query_start_loc, h_seq_lens, num_requests, block_size, &max_pages);
  if (st != CB_OK) return st;
  if (num_groups > 0) {
    if (h_group_start[0] != 0 || h_group_start[num_groups] != num_requests)
      return report_error(CB_ERR_METADATA, "h_group_start must run from 0 to num_requests");
    for (int g = 0; g < num_groups; ++g) {
      if (h_group_start[g + 1] < h_group_start[g] || h_group_start[g + 1] > num_requests)
        return report_error(CB_ERR_METADATA, "h_group_start must be non-decreasing");
      int32_t p = -1;
      for (int r = h_group_start[g]; r < h_group_start[g + 1]; ++r) {
        const int32_t ql = h_query_start_loc[r + 1] - h_query_start_loc[r];
        if (ql == 0) continue;
        if (p >= 0 && h_prefix_lens[r] != p)
          return report_error(CB_ERR_METADATA, "the requests of a group must have the same prefix length");
        p = h_prefix_lens[r];
        if (p < 0 || p % block_size != 0 || p > h_seq_lens[r] - ql)
          return report_error(CB_ERR_METADATA,
                              "a prefix must be whole blocks of every request's context");
        if (p > 0 && ql > 1)
          return report_error(CB_ERR_METADATA, "requests with q_len > 1 must have prefix length 0");
      }
    }
  }
  const cb::ScatterInputs rows{k_new, v_new, slot_mapping};
  if (num_tokens > 0 && num_groups > 0 && out && q && k_cache && v_cache && query_start_loc && seq_lens &&
      block_table && (!k_new || (v_new && slot_mapping)) && h_query_start_loc[num_requests] == num_tokens &&
      max_pages <= block_table_stride) {
    if (!prefix_lens) return report_error(CB_ERR_INVALID_ARG, "null pointer");
    for (const void* p : {(const void*)out, q, (const void*)k_cache, (const void*)v_cache, k_new, v_new,
                          (const void*)workspace})
      if (!cb::is_aligned16(p))
        return report_error(CB_ERR_INVALID_ARG, "q/out/K/V/workspace pointers must be 16-byte aligned");
    cb::StepArgs a = {};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.query_start_loc = query_start_loc;
    a.seq_lens = seq_lens;
    a.block_table = block_table;
    a.bt_stride = block_table_stride;
    a.num_requests = num_requests;
    a.num_tokens = num_tokens;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)head_dim)) * 1.4426950408889634f;
    a.sliding_window = sliding_window > 0 ? sliding_window : 0;
    a.dtype = dtype;
    a.test_expire_wait = (flags & CB_FLAG_TEST_WAIT_EXPIRY) ? 1 : 0;
    a.error_word = static_cast<int32_t*>(workspace);
    a.kv_start = prefix_lens;
    static thread_local SharedPlan sp;  // its vectors keep their storage from call to call
    if (plan_shared(sp, a, h_query_start_loc, h_seq_lens, h_prefix_lens, h_group_start, num_groups, flags,
                    k_new ? &rows : nullptr, workspace, workspace_bytes)) {
      const cudaError_t e = run_shared(sp, a, k_new ? &rows : nullptr, static_cast<cudaStream_t>(stream));
      return e == cudaSuccess ? CB_OK : cb::report_cuda_error(e, "shared-prefix attention launch");
    }
  }
  // no group worth sharing, or a shape of the portable kernels: the plain step reads the aliased
  // pages through every request's own block table (and reports what is malformed)
  return cb_paged_attention(out, q, k_cache, v_cache, k_new, v_new, slot_mapping, query_start_loc,
                            seq_lens, block_table, block_table_stride, h_query_start_loc, h_seq_lens,
                            num_requests, num_tokens, num_blocks, block_size, num_q_heads, num_kv_heads,
                            head_dim, scale, sliding_window, dtype, flags, workspace, workspace_bytes,
                            stream);
}

}  // namespace

extern "C" {

size_t cb_workspace_size_shared(int32_t num_requests, int32_t num_tokens, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim) {
  const size_t plain = cb_workspace_size(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim);
  if (num_requests < 0 || num_tokens < 0 || num_q_heads <= 0 || head_dim <= 0) return plain;
  return std::max(plain, shared_bytes(num_requests, num_tokens, num_q_heads, head_dim));
}

cb_status cb_paged_attention_shared(
    void* out, const void* q, void* k_cache, void* v_cache, const void* k_new, const void* v_new,
    const int64_t* slot_mapping, const int32_t* query_start_loc, const int32_t* seq_lens,
    const int32_t* block_table, int32_t block_table_stride, const int32_t* prefix_lens,
    const int32_t* h_query_start_loc, const int32_t* h_seq_lens, const int32_t* h_prefix_lens,
    const int32_t* h_group_start, int32_t num_groups, int32_t num_requests, int32_t num_tokens,
    int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, float scale, int32_t sliding_window, int32_t dtype, uint32_t flags,
    void* workspace, size_t workspace_bytes, void* stream) {
  try {
    return attention_shared(out, q, k_cache, v_cache, k_new, v_new, slot_mapping, query_start_loc,
                            seq_lens, block_table, block_table_stride, prefix_lens, h_query_start_loc,
                            h_seq_lens, h_prefix_lens, h_group_start, num_groups, num_requests,
                            num_tokens, num_blocks, block_size, num_q_heads, num_kv_heads, head_dim,
                            scale, sliding_window, dtype, flags, workspace, workspace_bytes, stream);
  } catch (...) {  // host memory ran out while planning; nothing was launched
    return report_error(CB_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"
