// Entry points of the 8-bit paged cache (declared in include/cb.h): validation, planning from
// the host mirrors and the launches of one step.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <climits>
#include <vector>

#include "api.h"
#include "cb.h"
#include "launch.h"
#include "merge.h"
#include "plan.h"
#include "q8.h"

namespace {

using cb::report_error;

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Requests of more query columns (tokens x grouped heads) than this are prefilled: their pages
// are turned into bf16 once and the tcgen05 tiles read those. Below it, and where they are small
// (small_run_blocks), the split kernel reads the 8-bit pages directly, once per item of up to 64
// columns (16 runs of 17 tokens behind 2000 positions, 32/8 heads: 76 us as chunks, 111 split).
constexpr int kChunkColumns = 64;

// How a CTA's consumer warps divide the work on items of up to `columns` query columns: 16 warps
// of 96 registers with 8 columns each, or 8 of 168 with 16.
struct Split {
  int column_blocks;  // NB: 8-column blocks per warp
  int column_warps;   // CW
  int heads;          // HB: KV heads per CTA, a divisor of Hkv
  int key_warps;      // KW
};

Split split_of(int64_t columns, int Hkv) {
  Split s;
  s.column_blocks = columns <= 8 ? 1 : 2;
  s.column_warps = 1;
  while (s.column_warps < cb::kQ8MaxColumnWarps && 16 * s.column_warps < columns) s.column_warps *= 2;
  const int warps = s.column_blocks == 1 ? 16 : 8;
  s.heads = std::min({Hkv, cb::kQ8MaxHeads, warps / s.column_warps});
  while (Hkv % s.heads != 0) --s.heads;
  s.key_warps = 1;
  while (2 * s.key_warps * s.heads * s.column_warps <= warps) s.key_warps *= 2;
  return s;
}

int tokens_per_item(const Split& s, int G) { return 8 * s.column_blocks * s.column_warps / G; }

// What a key block costs with items of 8, 16, 32 and 64 columns (64 requests of 128 .. 2048
// positions). From three KV heads on (32/8 heads of 128, runs of 2, 4, 8 and 16 tokens: 38.5, 41.8,
// 71.6 and 131.7 us, of which 9 are not the blocks') wider items convert the same keys in every
// column warp, so that they save little but the reading: a run of 10 tokens between 63 decode rows
// took 118 us as one item of 64 columns, and the decode rows with it, against 35 as five of 8. With
// one or two heads blocks are small and what they cost is their issue, once per item (8/1 heads of
// 128, runs of 8 tokens: 88, 50, 37 and 31 us with items of 8, 16, 32 and 64).
constexpr double kBlockCost[2][4] = {{1.0, 1.12, 2.13, 4.17}, {0.8, 1.12, 1.6, 2.3}};

// Longer runs of at most this many key blocks in items of 16 columns (all runs together) stay in the
// split kernel: ~12 us of its time, what the pages' copy and the start of the tiles take (one run of
// 17 tokens behind 2000 positions, 32/8 heads of 128: 22 us as a chunk, 15 here; behind 16000: 45 and
// 57; 20 tokens behind 1000 beside 63 decode rows: 53 and 35). Blocks of fewer or narrower heads
// cost less, but not in proportion: the two meet at ~2200 blocks of 1024 values, 5500 of 256, 9500 of
// 128 and 16000 of 64.
int64_t small_run_blocks(int Hkv, int D) { return (int64_t)(2200.0 * pow(1024.0 / ((double)Hkv * D), 0.7)); }

// Units that chunks are split into, at most (a second round of the SMs gains nothing that the first
// does not have); pieces of a row, at most; and what a unit costs (microseconds of one SM): a
// 128-key tile against its pair of query tiles, and its start and its rows' way out.
constexpr int kMaxChunkUnits = 2 * cb::kQ8TableCtas;
constexpr int kMaxChunkPieces = 64;
constexpr double kTileUs = 1.9, kUnitUs = 4.0;

// Workspace: header (as cb_paged_attention's), statistics and outputs of the partial rows, then
// the scratch of the prefilled requests (page table, K pages, V pages), whose sizes follow from
// each step's lengths.
struct Layout {
  size_t part_ml, part_o;    // of the split kernel
  size_t chunk_ml, chunk_o;  // of chunks whose keys are split
  size_t chunk_entries;      // (row, head) partial results there
  size_t scratch;
};

// chunks: whether the step (or the largest one) has requests that are prefilled.
Layout layout_of(int64_t R, int64_t T, int Hq, int Hkv, int D, bool chunks) {
  const int G = std::max(1, Hq / Hkv);
  int64_t rows = 0;  // (items + CTAs) x warps per head x tokens per item
  for (int columns = std::max(8, G); columns <= 16 * cb::kQ8MaxColumnWarps; columns *= 2) {
    const Split s = split_of(columns, Hkv);
    const int64_t TT = std::max(1, tokens_per_item(s, G));
    const int64_t C = std::max(1, cb::kQ8TableCtas / (Hkv / s.heads));
    rows = std::max(rows, ((T + R * (TT - 1)) / TT + R + C) * TT * s.key_warps);
  }
  Layout w;
  w.part_ml = cb::kWorkspaceHeaderBytes;
  w.part_o = w.part_ml + align256((size_t)rows * Hq * 8);
  w.chunk_ml = w.part_o + align256((size_t)rows * Hq * D * 4);
  // a unit has at most 256 (row, head) results
  w.chunk_entries =
      chunks ? (size_t)std::min<int64_t>((int64_t)kMaxChunkUnits * 256, T * Hq * kMaxChunkPieces) : 0;
  w.chunk_o = w.chunk_ml + align256(w.chunk_entries * 8);
  w.scratch = w.chunk_o + align256(w.chunk_entries * D * 4);
  return w;
}

size_t scratch_bytes(int64_t table_pages, int64_t pages, int block_size, int Hkv, int D) {
  return align256((size_t)table_pages * 4) + 2 * (size_t)pages * block_size * Hkv * D * 2;
}

// A request's query tokens that a CTA's warps take at once, and the key blocks they attend.
struct Item {
  int r, tile, blocks;
};

// What starting and finishing a piece of an item costs a CTA, in key blocks: its query rows, the
// first maximum, the partial rows (64 requests of 128 .. 2048 positions: CTAs with one piece were
// done after 23.1 us, with two after 25.9, with three after 28.7; a block takes 0.8).
constexpr int kPieceBlocks = 4;

struct Q8Plan {
  std::vector<Item> items;
  bool split = false;
  bool decode_only = false;  // every request has at most one query row
  int column_blocks = 1;
  cb::Q8Args args;
  std::vector<cb::MergeRow> merge;
  int max_pieces = 0;
  std::vector<cb::PrefillEntry> chunks;  // heaviest first
  int chunk_tiles = 0;                   // key tiles per unit of theirs (0: whole pairs)
  std::vector<cb::MergeRow> chunk_merge;
  int chunk_pieces = 0;
};

int first_key(int pos0, int window) { return window > 0 ? std::max(0, pos0 - window + 1) : 0; }

// Key blocks of the items of `tokens` query tokens of the requests with min_q <= q_len <= max_q, each
// item counted with `more` besides (up to `limit`).
int64_t split_blocks(const cb::StepArgs& a, const int32_t* qsl, const int32_t* seq_lens, int min_q, int max_q,
                     int tokens, int more, int64_t limit) {
  int64_t sum = 0;
  for (int r = 0; r < a.num_requests && sum <= limit; ++r) {
    const int q = qsl[r + 1] - qsl[r];
    if (q < min_q || q > max_q) continue;
    for (int t = 0; t < q && sum <= limit; t += tokens) {
      const int pos0 = seq_lens[r] - q + t, last = seq_lens[r] - q + std::min(q, t + tokens) - 1;
      sum += last / cb::kQ8KeyBlock - first_key(pos0, a.sliding_window) / cb::kQ8KeyBlock + 1 + more;
    }
  }
  return sum;
}

// The split kernel's launch over the requests with 1 <= q_len <= max_q.
void plan_split(Q8Plan& plan, const cb::StepArgs& a, const cb::Q8Cache& c, int max_q,
                const int32_t* qsl, const int32_t* seq_lens, const Layout& w, uint8_t* ws) {
  const int G = a.num_q_heads / a.num_kv_heads;
  int longest = 0;
  for (int r = 0; r < a.num_requests; ++r) {
    const int q = qsl[r + 1] - qsl[r];
    if (q <= max_q) longest = std::max(longest, q);
  }
  if (longest == 0) return;
  plan.split = true;
  plan.decode_only = longest == 1 && plan.chunks.empty();
  Split sp = {};
  double best = 0.0;
  for (int i = 0; i < 4; ++i) {  // the items' columns
    const int columns = 8 << i;
    if (columns < G) continue;
    const Split s = split_of(columns, a.num_kv_heads);
    const int64_t n = split_blocks(a, qsl, seq_lens, 1, max_q, columns / G, kPieceBlocks, INT64_MAX);
    const double cost = kBlockCost[a.num_kv_heads <= 2][i] * (double)n;
    if (best == 0.0 || cost < best) {
      best = cost;
      sp = s;
    }
    if (columns >= (int64_t)longest * G) break;
  }
  plan.column_blocks = sp.column_blocks;

  cb::Q8Args& p = plan.args;
  p.a = a;
  p.c = c;
  p.max_q = max_q;
  p.tile_tokens = tokens_per_item(sp, G);
  p.lg_group = 0;
  while ((1 << p.lg_group) < G) ++p.lg_group;
  p.lg_block = 0;
  while ((1 << p.lg_block) < a.block_size) ++p.lg_block;
  const int HB = p.heads_per_cta = sp.heads;
  p.column_warps = sp.column_warps;
  const int TT = p.tile_tokens, W = a.sliding_window;
  auto blocks = [&](int pos0, int ntok) {
    return (pos0 + ntok - 1) / cb::kQ8KeyBlock - first_key(pos0, W) / cb::kQ8KeyBlock + 1;
  };
  std::vector<Item>& items = plan.items;
  items.clear();
  long long U = 0;
  for (int r = 0; r < a.num_requests; ++r) {
    const int q = qsl[r + 1] - qsl[r];
    if (q < 1 || q > max_q) continue;
    for (int i = 0; i * TT < q; ++i) {
      const int pos0 = seq_lens[r] - q + i * TT, ntok = std::min(TT, q - i * TT);
      const int n = blocks(pos0, ntok);
      items.push_back(Item{r, i, n});
      U += n;
    }
  }
  const int groups = a.num_kv_heads / HB;
  long long C = std::max(1, std::min(cb::sm_count(), cb::kQ8TableCtas) / groups);
  C = std::min(C, (U + cb::kQ8MinBlocksPerCta - 1) / cb::kQ8MinBlocksPerCta);

  // fewer key warps (and partial rows) where each would have less than four blocks of a CTA's, one
  // where the CTAs have at most two each (16 requests of up to 300 positions: 7.5 us, 8.6 with two)
  p.key_warps = sp.key_warps;
  if (U <= 2 * C) p.key_warps = 1;
  while (p.key_warps > 2 && U < 4 * C * p.key_warps) p.key_warps /= 2;
  const int KW = p.key_warps;
  const int warps = HB * p.key_warps * p.column_warps;
  auto smem = [&](int stages) {
    return cb::q8_smem_bytes(a.head_dim, HB, warps, sp.column_blocks, a.dtype == CB_F32, stages, a.num_kv_heads);
  };
  const size_t fixed = smem(0), per = smem(1) - fixed;
  // each stage belongs to one producer and one key warp: whole multiples of both counts
  int m = std::max(p.key_warps, cb::kQ8Producers);
  p.stages = (int)std::min<size_t>(cb::kQ8MaxStages, cb::kQ8RingBytes / per) / m * m;
  if (p.stages * per < cb::kQ8RingBytes * 3 / 4 && p.stages + m <= cb::kQ8MaxStages &&
      fixed + (p.stages + m) * per <= (size_t)cb::kQ8SmemLimit)
    p.stages += m;
  // rings of many small blocks: groups of them, two groups per producer in the ring at least
  p.group_blocks = 1;
  while (p.group_blocks < 4 && p.stages % (4 * p.group_blocks * cb::kQ8Producers) == 0) p.group_blocks *= 2;

  // ---- the partition: CTAs are filled in order up to a load, the blocks they read and
  // kPieceBlocks for each piece they have; the least load (to a block) that C CTAs take
  auto fill = [&](long long load, auto&& piece) -> long long {  // CTAs used
    long long cta = 0, have = 0;
    for (size_t i = 0; i < items.size(); ++i) {
      int at = 0;
      while (at < items[i].blocks) {
        if (have + kPieceBlocks + 1 > load && have > 0) {
          ++cta;
          have = 0;
        }
        const int n = (int)std::min<long long>(items[i].blocks - at, std::max<long long>(1, load - have - kPieceBlocks));
        piece((int)cta, (int)i, at, n);
        have += kPieceBlocks + n;
        at += n;
      }
    }
    return cta + 1;
  };
  long long lo = (U + C - 1) / C + kPieceBlocks;  // no less
  long long hi = lo + (long long)kPieceBlocks * (long long)((items.size() + C - 1) / C + 1);
  auto nothing = [](int, int, int, int) {};
  while (fill(hi, nothing) > C) hi += hi - lo + 1;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (fill(mid, nothing) <= C) hi = mid; else lo = mid + 1;
  }
  int b0 = 0, last_cta = -1, u = 0, u0 = 0;
  fill(hi, [&](int cta, int i, int at, int n) {
    const Item& it = items[i];
    if (at == 0) {
      b0 = cta;
      u0 = u;
    }
    if (cta != last_cta) {
      p.start[cta] = cb::Q8CtaStart{u, it.r, it.tile, i, u0, qsl[it.r], qsl[it.r + 1] - qsl[it.r], seq_lens[it.r]};
      last_cta = cta;
    }
    u += n;
    const int pieces = (cta - b0 + 1) * KW;
    if (at + n == it.blocks && pieces > 1) {
      const int t0 = qsl[it.r] + it.tile * TT, ntok = std::min(TT, qsl[it.r + 1] - t0);
      for (int k = 0; k < ntok; ++k)
        plan.merge.push_back(cb::MergeRow{t0 + k, (i + b0) * KW * TT + k, TT, pieces, 0, 0, 0});
      plan.max_pieces = std::max(plan.max_pieces, pieces);
    }
  });
  C = last_cta + 1;
  p.num_ctas = (int)C;
  p.start[C] = cb::Q8CtaStart{(int)U, -1, 0, 0, 0, 0, 0, 0};
  p.k_new = p.v_new = nullptr;
  p.slot_mapping = nullptr;
  p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
}

// Bytes the prefilled requests need behind the partial rows; fills plan.chunks.
size_t plan_chunks(Q8Plan& plan, const cb::StepArgs& a, int max_q, const int32_t* qsl,
                   const int32_t* seq_lens) {
  const int TQ = 128 / (a.num_q_heads / a.num_kv_heads);
  int64_t pages = 0, table = 0;
  for (int r = 0; r < a.num_requests; ++r) {
    const int q = qsl[r + 1] - qsl[r];
    if (q <= max_q) continue;
    plan.chunks.push_back(cb::PrefillEntry{r, (q + TQ - 1) / TQ, qsl[r], q, seq_lens[r]});
    const int64_t all = ((int64_t)seq_lens[r] + a.block_size - 1) / a.block_size;
    table += all;
    pages += all - first_key(seq_lens[r] - q, a.sliding_window) / 128 * 128 / a.block_size;
  }
  if (plan.chunks.empty()) return 0;
  std::stable_sort(plan.chunks.begin(), plan.chunks.end(), [](const auto& x, const auto& y) {
    return (long long)x.seq_len * x.q_len > (long long)y.seq_len * y.q_len;
  });
  return scratch_bytes(table, pages, a.block_size, a.num_kv_heads, a.head_dim);
}

// Key tiles that a pair of a chunk's query tiles attends.
int pair_tiles(const cb::PrefillEntry& e, int pair, int TQ, int window) {
  const int ctx = e.seq_len - e.q_len, tok0 = 2 * pair * TQ, end = std::min(e.q_len, tok0 + 2 * TQ);
  return (ctx + end - 1) / 128 - first_key(ctx + tok0, window) / 128 + 1;
}

// Pieces that the keys of an entry's longest pair are split into.
int entry_splits(const cb::PrefillEntry& e, int TQ, int window, int per) {
  int splits = 1;
  for (int p = 0; 2 * p < e.n_qtiles; ++p)
    splits = std::max(splits, (pair_tiles(e, p, TQ, window) + per - 1) / per);
  return splits;
}

// Whether and how far the chunks' keys are split. Whole pairs take no merge, but leave SMs idle
// where there are few of them: the longest pair is the time while they are no more than the SMs.
// Otherwise all units' time over the SMs and half a unit for the uneven end; for a split also the
// partial rows written and read again (about 4 TB/s) and the merge's launches. The least time is
// taken, a split only where it gains a tenth.
void split_chunks(Q8Plan& plan, const cb::StepArgs& a, size_t max_entries) {
  const int TQ = 128 / (a.num_q_heads / a.num_kv_heads), W = a.sliding_window, S = cb::sm_count();
  long long pairs = 0, tiles = 0;
  int longest = 1;
  for (const cb::PrefillEntry& e : plan.chunks)
    for (int p = 0; 2 * p < e.n_qtiles; ++p) {
      const int n = pair_tiles(e, p, TQ, W);
      longest = std::max(longest, n);
      tiles += n;
      ++pairs;
    }
  auto time = [&](long long units, int per) {
    const double unit = per * kTileUs + kUnitUs;
    if (units * a.num_kv_heads <= S) return unit;
    return std::max(unit, (tiles * kTileUs + units * kUnitUs) * a.num_kv_heads / S + 0.5 * unit);
  };
  double best = 0.9 * time(pairs, longest);
  for (int k = 2; k <= kMaxChunkPieces && k <= longest; ++k) {  // pieces of the longest pair
    const int per = (longest + k - 1) / k;
    if (pairs * a.num_kv_heads * (k - 1) > kMaxChunkUnits) break;
    long long units = 0, rows = 0;
    for (const cb::PrefillEntry& e : plan.chunks) {
      const int splits = entry_splits(e, TQ, W, per);
      if (splits > 1) rows += (long long)splits * e.q_len;
      for (int p = 0; 2 * p < e.n_qtiles; ++p) units += (pair_tiles(e, p, TQ, W) + per - 1) / per;
    }
    const double t = time(units, per) + (double)rows * a.num_q_heads * a.head_dim * 8 / 4e6 +
                     3.0 * (double)((a.num_tokens + 1023) / 1024);
    if ((size_t)rows * a.num_q_heads <= max_entries && t < best) {
      best = t;
      plan.chunk_tiles = per;
    }
  }
}

// The prefilled requests, up to kPrefillMaxEntries a launch: their pages as bf16, the tiles, and
// the merge of the rows whose keys were split.
cudaError_t run_chunks(Q8Plan& plan, const cb::StepArgs& a, const cb::Q8Cache& c, const Layout& w,
                       uint8_t* ws, cudaStream_t s) {
  int64_t table = 0, total = 0;
  for (const cb::PrefillEntry& e : plan.chunks) {
    const int64_t all = ((int64_t)e.seq_len + a.block_size - 1) / a.block_size;
    table += all;
    total += all - first_key(e.seq_len - e.q_len, a.sliding_window) / 128 * 128 / a.block_size;
  }
  uint8_t* scratch = ws + w.scratch;
  uint8_t* k = scratch + align256((size_t)table * 4);
  uint8_t* v = k + (size_t)total * a.block_size * a.num_kv_heads * a.head_dim * 2;
  const int TQ = 128 / (a.num_q_heads / a.num_kv_heads), per = plan.chunk_tiles;
  int row = 0, dst = 0, part = 0;
  static thread_local cb::DequantArgs d;
  static thread_local cb::PrefixArgs pa;
  for (size_t i = 0; i < plan.chunks.size(); i += cb::kPrefillMaxEntries) {
    const int n = (int)std::min<size_t>(cb::kPrefillMaxEntries, plan.chunks.size() - i);
    d.c = c;
    d.block_table = a.block_table;
    d.bt_stride = a.bt_stride;
    d.num_blocks = a.num_blocks;
    d.block_size = a.block_size;
    d.num_kv_heads = a.num_kv_heads;
    d.head_dim = a.head_dim;
    d.k = k;
    d.v = v;
    d.table = reinterpret_cast<int32_t*>(scratch);
    d.error_word = a.error_word;
    d.dst0 = dst;
    static_cast<cb::PrefillArgs&>(pa) = cb::PrefillArgs{};
    pa.a = a;
    pa.a.k_cache = k;
    pa.a.v_cache = v;
    pa.a.block_table = d.table;
    pa.a.bt_stride = 1;  // an entry's "request" is the offset of its table row
    pa.a.num_blocks = (int)total;
    pa.tile_tokens = TQ;
    pa.box_keys = std::min(a.block_size, 128);
    pa.metadata_ready = 1;
    int* header = a.error_word;  // the workspace's first word
    pa.exit_counter = header + cb::kExitCounterOffset / 4;
    pa.unit_counter = header + cb::kUnitCounterOffset / 4;
    pa.scatter_counter = header + cb::kScatterCounterOffset / 4;
    pa.tiles_per_unit = per;  // (0: none of these are read)
    pa.part_ml = reinterpret_cast<float2*>(ws + w.chunk_ml);
    pa.part_o = reinterpret_cast<float*>(ws + w.chunk_o);
    for (int j = 0; j < n; ++j) {
      cb::PrefillEntry e = plan.chunks[i + j];
      const int all = (e.seq_len + a.block_size - 1) / a.block_size;
      const int first_pos = first_key(e.seq_len - e.q_len, a.sliding_window);
      const int first = first_pos / 128 * 128 / a.block_size;
      d.entries[j] = cb::DequantEntry{e.r, first, all - first, dst, row, first_pos};
      int splits = 1;
      if (per > 0) {
        splits = entry_splits(e, TQ, a.sliding_window, per);
        pa.splits[j] = splits;
        pa.part_row[j] = part;
        for (int p = 0; 2 * p < e.n_qtiles; ++p) {
          const int pieces = (pair_tiles(e, p, TQ, a.sliding_window) + per - 1) / per;
          if (pieces == 1) continue;  // written directly
          for (int t = 2 * p * TQ; t < std::min(e.q_len, 2 * (p + 1) * TQ); ++t)
            plan.chunk_merge.push_back(cb::MergeRow{e.q_start + t, part + t, e.q_len, pieces, 0, 0, 0});
          plan.chunk_pieces = std::max(plan.chunk_pieces, pieces);
        }
        if (splits > 1) part += splits * e.q_len;
      }
      e.r = row;
      pa.entries[j] = e;
      pa.total_units += (e.n_qtiles + 1) / 2 * a.num_kv_heads * splits;
      row += all;
      dst += all - first;
    }
    d.n_entries = pa.n_entries = n;
    d.n_pages = dst - d.dst0;
    pa.total_ctas = pa.total_units;
    pa.grid = std::min(pa.total_units, cb::sm_count());
    cudaError_t e = cb::launch_dequant_pages_q8(d, s);
    if (e == cudaSuccess) e = per > 0 ? cb::launch_split_chunks(pa, s) : cb::launch_prefill(pa, s);
    if (e != cudaSuccess) return e;
  }
  if (plan.chunk_merge.empty()) return cudaSuccess;
  cb::MergeArgs m;
  m.out = a.out;
  m.dtype = a.dtype;
  m.num_q_heads = a.num_q_heads;
  m.head_dim = a.head_dim;
  m.part_o = pa.part_o;
  m.part_ml = pa.part_ml;
  m.parts = cb::merge_parts(plan.chunk_pieces);
  return cb::launch_merge(m, plan.chunk_merge.data(), (int)plan.chunk_merge.size(), s);
}

cb_status check_rows(const void* k, const void* v, const cb::Q8Cache& c,
                     const int64_t* slot_mapping, int32_t num_tokens, int32_t num_blocks,
                     int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                     bool* empty) {
  *empty = false;
  if (dtype != CB_F32 && dtype != CB_BF16)
    return report_error(CB_ERR_INVALID_ARG, "dtype must be CB_F32 or CB_BF16");
  if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return report_error(CB_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (head_dim != 64 && head_dim != 128)
    return report_error(CB_ERR_UNSUPPORTED, "8-bit cache: head_dim must be 64 or 128");
  if ((int64_t)num_tokens * num_kv_heads >= (int64_t)1 << 33)
    return report_error(CB_ERR_UNSUPPORTED, "8-bit cache: too many rows in one call");
  if (num_tokens == 0) {
    *empty = true;
    return CB_OK;
  }
  if (!k || !v || !c.k || !c.v || !c.k_scale || !c.v_scale || !slot_mapping)
    return report_error(CB_ERR_INVALID_ARG, "null pointer");
  for (const void* p : {k, v, (const void*)c.k, (const void*)c.v, (const void*)c.k_scale,
                        (const void*)c.v_scale})
    if (!cb::is_aligned16(p))
      return report_error(CB_ERR_INVALID_ARG, "K/V and scale pointers must be 16-byte aligned");
  return CB_OK;
}

cb::Q8Cache cache_of(const void* k, const void* v, const void* ks, const void* vs) {
  auto u8 = [](const void* p) { return static_cast<uint8_t*>(const_cast<void*>(p)); };
  return cb::Q8Cache{u8(k), u8(v), u8(ks), u8(vs)};
}

cb_status attention_q8(void* out, const void* q, const cb::Q8Cache& c, const void* k_new,
                       const void* v_new, const int64_t* slot_mapping,
                       const int32_t* query_start_loc, const int32_t* seq_lens,
                       const int32_t* block_table, int32_t block_table_stride,
                       const int32_t* h_query_start_loc, const int32_t* h_seq_lens,
                       int32_t num_requests, int32_t num_tokens, int32_t num_blocks,
                       int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t head_dim, float scale, int32_t sliding_window, int32_t dtype,
                       uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
  cb_status st = cb::check_step_sizes(num_requests, num_tokens, num_blocks, block_size, num_q_heads,
                                      num_kv_heads, head_dim, block_table_stride, dtype,
                                      h_query_start_loc, h_seq_lens);
  if (st != CB_OK) return st;
  Layout w = layout_of(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim, false);
  if (!workspace || workspace_bytes < w.scratch + cb::kWorkspaceAlign)
    return report_error(CB_ERR_WORKSPACE, "workspace missing or smaller than cb_workspace_size_q8()");
  if (!cb::is_aligned16(workspace))
    return report_error(CB_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  int64_t max_pages = 0;
  st = cb::check_step_mirrors(h_query_start_loc, h_seq_lens, num_requests, block_size, &max_pages);
  if (st != CB_OK) return st;
  if (h_query_start_loc[num_requests] != num_tokens)
    return report_error(CB_ERR_METADATA, "query_start_loc[R] must equal num_tokens");
  if (max_pages > block_table_stride)
    return report_error(CB_ERR_METADATA,
                        "block_table_stride is smaller than ceil(seq_len / block_size)");
  if (num_tokens == 0) return CB_OK;
  if (!out || !q || !c.k || !c.v || !c.k_scale || !c.v_scale || !query_start_loc || !seq_lens ||
      !block_table)
    return report_error(CB_ERR_INVALID_ARG, "null pointer");
  if (k_new && (!v_new || !slot_mapping))
    return report_error(CB_ERR_INVALID_ARG, "k_new given without v_new or slot_mapping");
  for (const void* p : {(const void*)out, q, (const void*)c.k, (const void*)c.v,
                        (const void*)c.k_scale, (const void*)c.v_scale, k_new, v_new})
    if (!cb::is_aligned16(p))
      return report_error(CB_ERR_INVALID_ARG, "q/out/K/V/scale pointers must be 16-byte aligned");

  cb::StepArgs a = {};
  a.out = out;
  a.q = q;
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
  a.error_word = static_cast<int32_t*>(workspace);

  // a 16-key block lies in one page, or in two of 8 keys, whose scales are copied in multiples of 16
  // bytes; the rest runs on the portable kernel (which also takes head counts whose blocks' scales
  // would fill the ring)
  const bool fast = (block_size >= cb::kQ8KeyBlock || (block_size == 8 && num_kv_heads % 2 == 0)) &&
                    num_kv_heads <= 128 && !(flags & CB_FLAG_PORTABLE_ONLY);
  uint8_t* ws = cb::align_workspace(workspace);
  workspace_bytes -= cb::kWorkspaceAlign;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local Q8Plan plan;  // its vectors keep their storage from call to call
  plan.split = false;
  plan.merge.clear();
  plan.chunks.clear();
  plan.chunk_merge.clear();
  plan.chunk_tiles = plan.chunk_pieces = 0;
  plan.max_pieces = 0;
  if (fast) {
    const int G = num_q_heads / num_kv_heads;
    int max_q = dtype == CB_F32 ? INT_MAX : std::max(1, kChunkColumns / G);
    const size_t need = plan_chunks(plan, a, max_q, h_query_start_loc, h_seq_lens);
    if (need > 0) w = layout_of(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim, true);
    if (w.scratch > workspace_bytes || need > workspace_bytes - w.scratch)
      return report_error(CB_ERR_WORKSPACE,
                          "workspace too small for the step's chunks: chunk_kv_tokens of "
                          "cb_workspace_size_q8() must cover the seq_lens of requests with q_len > 1");
    if (need > 0) {
      const int64_t limit = small_run_blocks(num_kv_heads, head_dim);
      if (split_blocks(a, h_query_start_loc, h_seq_lens, max_q + 1, INT_MAX, 16 / G, 0, limit) <= limit) {
        plan.chunks.clear();
        max_q = INT_MAX;
      } else {
        split_chunks(plan, a, w.chunk_entries);
      }
    }
    plan_split(plan, a, c, max_q, h_query_start_loc, h_seq_lens, w, ws);
  }
  cudaError_t e = cudaSuccess;
  if (k_new && fast && plan.split && plan.decode_only) {
    plan.args.k_new = k_new;
    plan.args.v_new = v_new;
    plan.args.slot_mapping = slot_mapping;
  } else if (k_new) {
    e = cb::launch_write_kv_q8(k_new, v_new, c, slot_mapping, num_tokens,
                               (int64_t)num_blocks * block_size, num_kv_heads, head_dim, dtype,
                               a.error_word, s);
  }
  if (e != cudaSuccess) return cb::report_cuda_error(e, "write_kv_q8 launch");
  if (!fast) {
    e = cb::launch_q8_portable(a, c, s);
  } else {
    if (plan.split) e = cb::launch_q8_split(plan.args, plan.column_blocks, s);
    if (e == cudaSuccess && !plan.merge.empty()) {
      cb::MergeArgs m;
      m.out = out;
      m.dtype = dtype;
      m.num_q_heads = num_q_heads;
      m.head_dim = head_dim;
      m.part_o = plan.args.part_o;
      m.part_ml = plan.args.part_ml;
      m.parts = cb::merge_parts(plan.max_pieces);
      e = cb::launch_merge(m, plan.merge.data(), (int)plan.merge.size(), s);
    }
    if (e == cudaSuccess && !plan.chunks.empty()) e = run_chunks(plan, a, c, w, ws, s);
  }
  if (e != cudaSuccess) return cb::report_cuda_error(e, "8-bit attention launch");
  return CB_OK;
}

}  // namespace

extern "C" {

cb_status cb_write_kv_q8(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         void* k_scale, void* v_scale, const int64_t* slot_mapping,
                         int32_t num_tokens, int32_t num_blocks, int32_t block_size,
                         int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                         int32_t* error_word, void* stream) {
  const cb::Q8Cache c = cache_of(k_cache, v_cache, k_scale, v_scale);
  bool empty = false;
  const cb_status st = check_rows(k_new, v_new, c, slot_mapping, num_tokens, num_blocks,
                                  block_size, num_kv_heads, head_dim, dtype, &empty);
  if (st != CB_OK || empty) return st;
  const cudaError_t e = cb::launch_write_kv_q8(
      k_new, v_new, c, slot_mapping, num_tokens, (int64_t)num_blocks * block_size, num_kv_heads,
      head_dim, dtype, error_word, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CB_OK : cb::report_cuda_error(e, "write_kv_q8 launch");
}

cb_status cb_read_kv_q8(const void* k_cache, const void* v_cache, const void* k_scale,
                        const void* v_scale, const int64_t* slot_mapping, void* k_out,
                        void* v_out, int32_t num_tokens, int32_t num_blocks, int32_t block_size,
                        int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                        int32_t* error_word, void* stream) {
  const cb::Q8Cache c = cache_of(k_cache, v_cache, k_scale, v_scale);
  bool empty = false;
  const cb_status st = check_rows(k_out, v_out, c, slot_mapping, num_tokens, num_blocks,
                                  block_size, num_kv_heads, head_dim, dtype, &empty);
  if (st != CB_OK || empty) return st;
  const cudaError_t e = cb::launch_read_kv_q8(
      k_out, v_out, c, slot_mapping, num_tokens, (int64_t)num_blocks * block_size, num_kv_heads,
      head_dim, dtype, error_word, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CB_OK : cb::report_cuda_error(e, "read_kv_q8 launch");
}

size_t cb_workspace_size_q8(int32_t num_requests, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t chunk_kv_tokens) {
  if (num_requests < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0)
    return cb::kWorkspaceHeaderBytes;
  const size_t fixed = layout_of(num_requests, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                 chunk_kv_tokens > 0).scratch + cb::kWorkspaceAlign;
  if (chunk_kv_tokens <= 0) return fixed;
  // each request's pages are rounded up
  const int64_t pages = chunk_kv_tokens / block_size + std::min<int64_t>(num_requests, chunk_kv_tokens);
  return fixed + scratch_bytes(pages, pages, block_size, num_kv_heads, head_dim);
}

cb_status cb_paged_attention_q8(void* out, const void* q, void* k_cache, void* v_cache,
                                void* k_scale, void* v_scale, const void* k_new,
                                const void* v_new, const int64_t* slot_mapping,
                                const int32_t* query_start_loc, const int32_t* seq_lens,
                                const int32_t* block_table, int32_t block_table_stride,
                                const int32_t* h_query_start_loc, const int32_t* h_seq_lens,
                                int32_t num_requests, int32_t num_tokens, int32_t num_blocks,
                                int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, float scale, int32_t sliding_window,
                                int32_t dtype, uint32_t flags, void* workspace,
                                size_t workspace_bytes, void* stream) {
  try {
    return attention_q8(out, q, cache_of(k_cache, v_cache, k_scale, v_scale), k_new, v_new,
                        slot_mapping, query_start_loc, seq_lens, block_table, block_table_stride,
                        h_query_start_loc, h_seq_lens, num_requests, num_tokens, num_blocks,
                        block_size, num_q_heads, num_kv_heads, head_dim, scale, sliding_window,
                        dtype, flags, workspace, workspace_bytes, stream);
  } catch (...) {  // host memory ran out while planning (some of the step may be launched)
    return report_error(CB_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"
