// Attention over the 8-bit paged cache (q8.cuh): split-KV kernel for decode rows and short
// runs of query tokens, and a portable CUDA-core kernel for the shapes it does not cover.
//
// Split kernel. What it computes is the per-block pseudocode of "Continuous Batching"
// (languisher.top), section "Extension: the vLLM v1 implementation", on rows that stand in the
// cache as y * 2^e. With the K row's exponent ek, the V row's ev and column c (a query token
// and head of the KV head's group):
//     s_j = scale_log2 <q_c, yk_j> 2^ek_j          (log2 units)
//     out_c = sum_j 2^s_j 2^ev_j yv_j / sum_j 2^s_j
// so both scales leave the contractions: 2^ek multiplies a score, ev is added to the exponent
// of the weight that multiplies V.
//
// Decode streams every attended byte once and is HBM-bound, now at half the bytes of a bf16
// cache; the kernel must turn each byte into a tensor-core operand at ~44 bytes/ns per SM.
//
// * Partition. The (request, tile of query tokens) items' 16-key blocks are numbered in
//   request order and CTA b of C takes blocks [b U / C, (b + 1) U / C): equal bytes per CTA.
//   Each warp's share of an item in a CTA (a piece) becomes a partial row that the merge kernel
//   joins (merge.h); only an item that one warp per head has to itself is written directly.
// * Staging. Producer warps bring each block (16 keys, up to 8 KV heads, K and V) with two
//   swizzled tensor copies (four where a page has 8 keys), and its scales with two bulk copies, into a ring of stages. One
//   warp needs ~0.5 us to place and issue a block, which bounded everything but the widest
//   rows: four warps take the blocks in turn, and where blocks are small several lanes of
//   each a block of their own at once.
// * Operands. e4m3 is exact in fp16, so the contractions are fp16 mma.sync with fp32
//   accumulation, and the conversion is one instruction per pair (cvt.f16x2.e4m3x2). q is
//   scaled per row by a power of two to a largest magnitude in [2^13, 2^14): a bf16 row is
//   then exact down to 2^-38 of its largest element, and an fp32 row is the sum of two fp16
//   rows to 2^-22. Weights are fp16 (bf16 queries: 11 bits, finer than the bf16 the output is
//   rounded to) or the sum of two fp16 (fp32 queries), scaled to at most 2^14 and, with the
//   maximum just raised, 2^6: the smallest are rounded to 2^-25, 2^-31 of the largest.
// * Layout. Keys are the M = 16 rows of both products' A operand side, columns the N = 8.
//   The contraction index may be permuted freely, so a lane takes its operands from whole
//   16-byte pieces of the staged rows: for S^T = K Q^T lane (g, t) holds d = D/4 t ..
//   D/4 t + D/4 - 1 of keys g and g + 8; for O^T = V^T P^T it holds d = D/8 g .. of keys
//   2t, 2t+1, 2t+8, 2t+9, pairs of keys interleaved bytewise (prmt) before the conversion.
//   O then has a lane's outputs contiguous in d: 32-byte stores.
// * Softmax. Two running maxima per column, of s_j (for the sum) and of s_j + ev_j (for the
//   weights), because rows of very different V scales may meet: with one maximum a large
//   scale on an unattended key would push the attended ones' weights under fp16's range. Both
//   are raised only when exceeded by more than 2^8, which a warp vote finds without the
//   cross-lane maximum. Statistics, sums and outputs are fp32.
// * Warps. KW warps share a KV head and take the blocks in turn, each with its own state and its
//   own partial rows: a join through shared memory at the end of each piece cost 1.5 us there,
//   in which the stream stood still, and the merge kernel has to run anyway. At 8 heads and two
//   warps each, one warp has ~1400 cycles per 16-key block at the HBM rate. Runs of query tokens
//   have up to 64 columns: CW warps of a head then read the same blocks for 16 columns each (the
//   CTA has that many fewer heads), so that the cache is still read once; or the run is several
//   items of fewer columns, which read it again (the planner chooses per step).
// Measured (32/8 heads of 128 unless said): 16 requests of 32768 positions, 64/8 heads: 162 us, 98 %
// of the copy rate; 64 requests of 128 .. 2048: 30.4 us for 141 MB, of which ~8 us are start, pieces'
// ends and merge; the same with runs of 4 tokens 41.8 us, fp32 55.8; 4 requests of up to 301: 7.3 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <float.h>
#include <limits.h>

#include "cb.h"
#include "common.cuh"
#include "launch.h"
#include "q8.cuh"
#include "q8.h"
#include "sm100_ptx.cuh"

namespace cb {

namespace {

constexpr int kKB = kQ8KeyBlock;
constexpr float kNoMax = -1e30f;     // running maximum before any key (finite: no inf - inf)
constexpr float kRaise = 8.f;        // the maxima are raised when exceeded by more than 2^8
constexpr float kWeightLog2 = 6.f;   // weights are at most 2^(8 + 6), inside fp16's range
constexpr int kQueue = 4;            // pieces handed ahead to the consumers

struct Q8Piece {
  int r;       // request
  int t0;      // packed query row of the item's first token (-1: no more pieces)
  int ntok;
  int n;       // key blocks of this piece
  int kb0;     // first of them
  int pos0;    // position of the first token
  int slot;    // partial slot (item + CTA)
  int direct;  // the whole item is one warp's per head
  int last;    // the piece ends with the item's last key block
};

// The new row of the request whose last block a consumer warp is going to read, quantised.
struct Q8NewRow {
  uint32_t k[32], v[32];  // D / 4 words each
  int k_code, v_code;
  long long row;          // its row in the cache (slot * Hkv + head), -1: not written
  int staged;             // its slot is its own position's: it is attended as well
};

struct Q8Smem {
  uint64_t full[kQ8MaxStages];
  uint64_t empty[kQ8MaxStages];
  uint64_t pfull[kQueue];
  uint64_t pempty[kQueue];
  Q8Piece piece[kQueue];
  Q8NewRow fresh[16];  // by consumer warp: the warps of a head may be pieces apart
  int abort_flag;
};

// Bytes of a warp's query fragments. They stay in shared memory: in registers they made the key
// loop spill (16 of 96 registers, twice that for fp32 queries).
__host__ __device__ constexpr int q_frag_bytes(int D, int NB, bool f32) {
  return D / 16 * NB * (f32 ? 2 : 1) * 256;
}

// Position of key row i (0 .. 15) of a tile within its block. For D 64 (64-byte rows) the low
// two bits change places, so that the rows of a V fragment (2t, t = 0 .. 3) fall on both
// halves of the banks.
template <int D>
CB_DEV int key_of_row(int i) {
  return D == 64 ? ((i & ~3) | ((i & 1) << 1) | ((i & 2) >> 1)) : i;
}

// Byte offset of 16-byte chunk c of staged row `row` (rows of D bytes, copied with the 128- or
// 64-byte swizzle).
template <int D>
CB_DEV uint32_t row_chunk(int row, int c) {
  if constexpr (D == 128) return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4));
  return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

CB_DEV void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

CB_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The pair's remainder after rounding to fp16, as fp16.
CB_DEV uint32_t pack_f16x2_rest(uint32_t rounded, float lo, float hi) {
  const float2 r = float2_of_f16x2(rounded);
  return pack_f16x2(lo - r.x, hi - r.y);
}

CB_DEV uint32_t f16x2_lo(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)w); }
CB_DEV uint32_t f16x2_hi(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)(w >> 16)); }

// Ask for the line of `p` in L1 (a hint).
CB_DEV void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// A operand of O^T = V^T P^T for two output tiles of head_dim: words of four V rows (keys 2t, 2t+1,
// 2t+8, 2t+9), the bytes of a pair of keys side by side (bytes 0, 1 of the words, or 2, 3).
CB_DEV void v_fragment(uint32_t (&a)[4], uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, bool hi) {
  const uint32_t sel = hi ? 0x7362u : 0x5140u;
  const uint32_t x = __byte_perm(v0, v1, sel), y = __byte_perm(v2, v3, sel);
  a[0] = f16x2_lo(x);
  a[1] = f16x2_hi(x);
  a[2] = f16x2_lo(y);
  a[3] = f16x2_hi(y);
}

// 0xff in the bytes that are e4m3 NaNs, else 0.
CB_DEV uint32_t nan_bytes(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }

CB_DEV uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

CB_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

CB_DEV int lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return (int)v;
}

CB_DEV void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
CB_DEV void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
CB_DEV void sts8(uint32_t addr, int v) {
  asm volatile("st.shared.b8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Four values of a row (16-byte aligned fp32, 8-byte aligned bf16), their largest finite
// magnitude's bits, and their e4m3 bytes.
template <bool F32>
CB_DEV void load4(const void* rows, long long at, float (&x)[4]) {
  if constexpr (F32) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(rows) + at));
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(rows) + at));
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
CB_DEV uint32_t magnitude4(const float (&x)[4]) {
  return max(max(finite_magnitude(x[0]), finite_magnitude(x[1])),
             max(finite_magnitude(x[2]), finite_magnitude(x[3])));
}
CB_DEV uint32_t quantise4(const float (&x)[4], float inv) {
  return e4m3x2_of(x[0] * inv, x[1] * inv) | (e4m3x2_of(x[2] * inv, x[3] * inv) << 16);
}

// First key block of a run of ntok tokens starting at position pos0, and how many it attends.
CB_DEV int first_key(int pos0, int window) { return window > 0 ? max(0, pos0 - window + 1) : 0; }
CB_DEV int blocks_of(int pos0, int ntok, int window) {
  return (pos0 + ntok - 1) / kKB - first_key(pos0, window) / kKB + 1;
}

}  // namespace

// NB column blocks of 8; F32: fp32 queries and outputs (operands split into two fp16 parts); P8: pages
// of 8 keys (an instance of its own: with the offsets as variables the others spilled 104 bytes
// instead of 76). 64 requests of 128 .. 2048 positions, 32/8 heads: 30.0 us in pages of 8 and 29.7 of
// 16; on the portable kernel 365.
template <int D, int NB, bool F32, bool P8>
__global__ void __launch_bounds__(((NB == 1 ? 16 : 8) + kQ8Producers) * 32, 1)
q8_split_kernel(const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ Q8Args p) {
  constexpr int kKS = D / 16;          // contraction steps over head_dim; output tiles of 16
  constexpr int kSplit = F32 ? 2 : 1;  // fp16 parts of q and of the weights
  extern __shared__ __align__(1024) uint8_t smem_dyn[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const int HB = p.heads_per_cta, KW = p.key_warps, CW = p.column_warps, Hkv = p.a.num_kv_heads;
  const int box_bytes = HB * kKB * D;      // K (or V) of one block
  const int stage_bytes = 2 * box_bytes;
  const int scale_bytes = kKB * Hkv;       // K (or V) scales of one block, every head
  uint8_t* stages = base;
  uint8_t* scales = stages + p.stages * stage_bytes;
  uint8_t* qfrags = scales + p.stages * 2 * scale_bytes;
  Q8Smem& sm = *reinterpret_cast<Q8Smem*>(qfrags + HB * KW * CW * q_frag_bytes(D, NB, F32));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const int hg = blockIdx.y;
  const int nwarps = HB * KW * CW;  // consumer warps; the producers follow
  const int W = p.a.sliding_window;
  const int TT = p.tile_tokens;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], HB * CW);
    }
    for (int s = 0; s < kQueue; ++s) {
      mbar_init(&sm.pfull[s], 1);
      mbar_init(&sm.pempty[s], nwarps);
    }
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  // scales of a block that was never copied (a page id out of range) read as the smallest
  for (int i = threadIdx.x; i < p.stages * 2 * scale_bytes / 4; i += blockDim.x)
    reinterpret_cast<uint32_t*>(scales)[i] = 0u;
  fence_proxy_async_smem();
  if (warp == nwarps && lane == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  grid_dependency_wait();
  allow_dependent_launch();
  __syncthreads();

  const int GB = p.group_blocks;  // a power of two
  const int producer = warp - nwarps;
  int issued_blocks = 0;  // producers: one past the last block whose copies this warp issued
  if (producer >= 0) {
    // =================================================== producer warps
    // All walk the same pieces; block i is issued by warp i / GB % kQ8Producers, lanes of it the GB
    // blocks of a group together, and the first also hands the pieces to the consumers.
    const int u_lo = p.start[b].u, u_hi = p.start[b + 1].u;
    const uint64_t policy = l2_policy_evict_first();  // the stream is read once
    const int BS = p.a.block_size;
    bool ok = true;
    int k = 0;  // pieces handed out
    int i = 0;  // blocks issued
    int s = 0, round = 0;  // i % stages, i / stages
    // Request metadata, 32 requests at a time (lane l: request wbase + l).
    int wbase = -1, w_t = 0, w_q = 0, w_seq = 0;
    auto load_window = [&](int r0) {
      wbase = r0;
      const int r = r0 + lane;
      w_t = w_q = w_seq = 0;
      if (r < p.a.num_requests) {
        w_t = __ldg(p.a.query_start_loc + r);
        w_q = __ldg(p.a.query_start_loc + r + 1) - w_t;
        w_seq = __ldg(p.a.seq_lens + r);
        if (w_q > p.max_q) w_q = 0;  // another kernel's rows
      }
    };
    auto next_request = [&](int r) -> int {  // the next request with rows, from r on
      while (r < p.a.num_requests) {
        if (wbase < 0 || r - wbase >= 32 || r < wbase) load_window(r);
        const unsigned m = __ballot_sync(0xffffffffu, w_q > 0 && wbase + lane >= r);
        if (m) return wbase + __ffs(m) - 1;
        r = wbase + 32;
      }
      return -1;
    };
    // the current item: its request's fields, its first block and its block count
    int r = p.start[b].r, tile = p.start[b].tile, item = p.start[b].item;
    int u0 = p.start[b].u0;
    int t0 = 0, qlen = 0, seq = 0, pos0 = 0, ntok = 0, nblk = 0, kb_lo = 0;
    auto set_item = [&]() {
      pos0 = seq - qlen + tile * TT;
      ntok = min(TT, qlen - tile * TT);
      kb_lo = first_key(pos0, W) / kKB;
      nblk = blocks_of(pos0, ntok, W);
    };
    auto set_request = [&]() {
      const int j = r - wbase;
      t0 = __shfl_sync(0xffffffffu, w_t, j);
      qlen = __shfl_sync(0xffffffffu, w_q, j);
      seq = __shfl_sync(0xffffffffu, w_seq, j);
    };
    // page ids of key blocks kb .. kb + n - 1 of the request (lane l: block kb + l); in pages of 8
    // keys, pages2 has those of the blocks' second halves (kNoPage: past the request)
    constexpr int kNoPage = INT_MIN;
    int pages2 = kNoPage;
    auto load_pages = [&](int rr, int kb, int n) -> int {
      const int32_t* bt = p.a.block_table + (long long)rr * p.a.bt_stride;
      if constexpr (P8)
        pages2 = lane < n && ((kb + lane) * kKB + BS) < seq ? __ldg(bt + ((kb + lane) * 2 + 1)) : kNoPage;
      return lane < n ? __ldg(bt + ((kb + lane) * kKB >> p.lg_block)) : 0;
    };
    // one lane: the copies of key block kb, in page pg, into stage st_i
    auto copy_block = [&](int kb, int pg, int pg2, int st_i) {
      const int key0 = (kb * kKB) & (BS - 1);
      uint64_t* const full = &sm.full[st_i];
      uint8_t* st = stages + st_i * stage_bytes;
      uint8_t* sc = scales + st_i * 2 * scale_bytes;
      const bool page_ok = pg >= 0 && pg < p.a.num_blocks;
      if constexpr (P8) {  // 8 keys of each head from either page, one half of the stage behind the other
        const bool ok2 = pg2 >= 0 && pg2 < p.a.num_blocks;
        if (!page_ok || (!ok2 && pg2 != kNoPage)) record_error(p.a.error_word, CB_DEVERR_BLOCK_ID);
        const uint32_t half = (uint32_t)scale_bytes / 2;
        mbar_arrive_expect_tx(full, (uint32_t)stage_bytes + 2 * half * ((page_ok ? 1 : 0) + (ok2 ? 1 : 0)));
        for (int h = 0; h < 2; ++h) {
          const bool ok_h = h == 0 ? page_ok : ok2;
          const int page = ok_h ? (h == 0 ? pg : pg2) : p.a.num_blocks;
          tma_load_4d_hint(st + h * (box_bytes / 2), &tmap_k, full, 0, 0, hg * HB, page, policy);
          tma_load_4d_hint(st + box_bytes + h * (box_bytes / 2), &tmap_v, full, 0, 0, hg * HB, page, policy);
          if (ok_h) {
            const long long at = ((long long)page << p.lg_block) * Hkv;
            bulk_load(sc + h * half, p.c.k_scale + at, half, full);
            bulk_load(sc + scale_bytes + h * half, p.c.v_scale + at, half, full);
          }
        }
        return;
      } else {
        if (!page_ok) record_error(p.a.error_word, CB_DEVERR_BLOCK_ID);
        mbar_arrive_expect_tx(full, (uint32_t)(stage_bytes + (page_ok ? 2 * scale_bytes : 0)));
        const int page = page_ok ? pg : p.a.num_blocks;  // past the pool: zeros
        tma_load_4d_hint(st, &tmap_k, full, 0, key0, hg * HB, page, policy);
        tma_load_4d_hint(st + box_bytes, &tmap_v, full, 0, key0, hg * HB, page, policy);
        if (page_ok) {
          const long long at = (((long long)pg << p.lg_block) + key0) * Hkv;
          bulk_load(sc, p.c.k_scale + at, (uint32_t)scale_bytes, full);
          bulk_load(sc + scale_bytes, p.c.v_scale + at, (uint32_t)scale_bytes, full);
        }
      }
    };
    bool more = u_lo < u_hi;
    int kb0 = 0, kb1 = 0, pages = 0;
    if (more) {
      // placed by the host: the first copies wait only for their page ids
      t0 = p.start[b].t0;
      qlen = p.start[b].q_len;
      seq = p.start[b].seq;
      set_item();
      kb0 = kb_lo + u_lo - u0;
      kb1 = kb_lo + min(u0 + nblk, u_hi) - u0;
      pages = load_pages(r, kb0, min(32, kb1 - kb0));
    }
    while (more && ok) {
      if (producer == 0) {
        const int qs = k % kQueue;
        if (k >= kQueue &&
            !mbar_wait_warp_or_abort(&sm.pempty[qs], (uint32_t)(k / kQueue - 1) & 1, &sm.abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          Q8Piece& d = sm.piece[qs];
          d.r = r;
          d.t0 = t0 + tile * TT;
          d.ntok = ntok;
          d.n = kb1 - kb0;
          d.kb0 = kb0;
          d.pos0 = pos0;
          d.slot = item + b;
          d.direct = KW == 1 && u0 >= u_lo && u0 + nblk <= u_hi;
          d.last = kb1 == kb_lo + nblk;
          mbar_arrive(&sm.pfull[qs]);
        }
        __syncwarp();
        {
          // the piece's query rows and new rows on their way into L1: under a full stream a load
          // takes over a microsecond, which the consumers would wait for at every piece
          const int elt = F32 ? 4 : 2, t = t0 + tile * TT;
          const uint8_t* q = static_cast<const uint8_t*>(p.a.q);
          const int row = p.a.num_q_heads * D * elt, part = (HB << p.lg_group) * D * elt;
          for (int i = lane * 128; i < ntok * part; i += 32 * 128)
            prefetch_l1(q + (long long)(t + i / part) * row + hg * part + i % part);
          if (p.k_new != nullptr && kb1 == kb_lo + nblk) {
            const long long at = ((long long)t * Hkv + hg * HB) * D * elt;
            for (int i = lane * 128; i < HB * D * elt; i += 32 * 128) {
              prefetch_l1(static_cast<const uint8_t*>(p.k_new) + at + i);
              prefetch_l1(static_cast<const uint8_t*>(p.v_new) + at + i);
            }
            if (lane == 0) prefetch_l1(p.slot_mapping + t);
            if (lane == 1) prefetch_l1(p.a.block_table + (long long)r * p.a.bt_stride + pos0 / BS);
          }
        }
      }
      ++k;
      // the item after this one, looked up once this piece's first copy is out
      bool looked = false;
      int nr = r, n_kb0 = 0, n_kb1 = 0;
      const int cur_r = r, first = kb0, last = kb1;
      const int u_end = u0 + nblk;
      for (int kb_base = first; kb_base < last && ok; kb_base += 32) {
        const int n = min(32, last - kb_base);
        const int cur = pages, cur2 = pages2;
        for (int j = 0, cnt; j < n; j += cnt) {
          if (GB == 1) {
            cnt = 1;
            if ((i & (kQ8Producers - 1)) == producer) {
              const int pg = __shfl_sync(0xffffffffu, cur, j);
              const int pg2 = P8 ? __shfl_sync(0xffffffffu, cur2, j) : kNoPage;
              if ((round > 0 &&
                   !mbar_wait_warp_or_abort(&sm.empty[s], (uint32_t)(round - 1) & 1, &sm.abort_flag)) ||
                  *reinterpret_cast<volatile int*>(&sm.abort_flag)) {
                ok = false;
                break;
              }
              if (lane == 0) copy_block(kb_base + j, pg, pg2, s);
              __syncwarp();
              issued_blocks = i + 1;
            }
          } else {
            cnt = min(GB - (i & (GB - 1)), n - j);  // blocks of this group
            if ((i / GB & (kQ8Producers - 1)) == producer) {
              // lane l < cnt: block j + l, stage s + l
              const int pg = __shfl_sync(0xffffffffu, cur, (j + lane) & 31);
              const int pg2 = P8 ? __shfl_sync(0xffffffffu, cur2, (j + lane) & 31) : kNoPage;
              const bool mine = lane < cnt;
              const bool free = !mine || round == 0 ||
                                mbar_wait_or_abort(&sm.empty[s + lane], (uint32_t)(round - 1) & 1, &sm.abort_flag);
              if (!__all_sync(0xffffffffu, free && *reinterpret_cast<volatile int*>(&sm.abort_flag) == 0)) {
                ok = false;
                break;
              }
              if (mine) copy_block(kb_base + j + lane, pg, pg2, s + lane);
              __syncwarp();
              issued_blocks = i + cnt;
            }
          }
          i += cnt;
          s += cnt;
          if (s == p.stages) {
            s = 0;
            ++round;
          }
          if (j == 0) {
            if (kb_base + 32 < last) {
              pages = load_pages(cur_r, kb_base + 32, min(32, last - kb_base - 32));
            } else if (!looked) {
              looked = true;
              more = u_end < u_hi;
              if (more) {
                if ((tile + 1) * TT < qlen) {
                  ++tile;
                } else {
                  tile = 0;
                  nr = next_request(r + 1);
                  if (nr < 0) {
                    more = false;
                  } else {
                    r = nr;
                    set_request();
                  }
                }
              }
              if (more) {
                ++item;
                u0 = u_end;
                set_item();
                n_kb0 = kb_lo;
                n_kb1 = kb_lo + min(u0 + nblk, u_hi) - u0;
                pages = load_pages(r, n_kb0, min(32, n_kb1 - n_kb0));
              }
            }
          }
        }
      }
      kb0 = n_kb0;
      kb1 = n_kb1;
    }
    if (ok && producer == 0) {
      const int qs = k % kQueue;
      if (k >= kQueue &&
          !mbar_wait_warp_or_abort(&sm.pempty[qs], (uint32_t)(k / kQueue - 1) & 1, &sm.abort_flag))
        ok = false;
      if (ok && lane == 0) {
        sm.piece[qs].t0 = -1;
        mbar_arrive(&sm.pfull[qs]);
      }
    }
    if (!ok && lane == 0) {
      record_error(p.a.error_word, CB_DEVERR_TIMEOUT);
      set_abort(&sm.abort_flag);
    }
  } else {
    // =================================================== consumer warps
    auto give_up = [&]() {
      if (lane == 0) {
        record_error(p.a.error_word, CB_DEVERR_TIMEOUT);
        set_abort(&sm.abort_flag);
      }
    };
    auto consume = [&]() {
      const int hl = warp % HB, kw = warp / HB % KW;
      const int col0 = warp / (HB * KW) * 8 * NB;  // this warp's columns of the item
      const int gid = lane >> 2, tq = lane & 3;
      const int G = 1 << p.lg_group;
      const int head = hg * HB + hl;  // KV head
      const int Hq = p.a.num_q_heads;
      const uint32_t stage0 = smem_u32(stages);
      const uint32_t scale0 = smem_u32(scales) + head;
      // This lane's pieces of a staged block. K: chunks of keys key_a and key_a + 8. V: keys
      // key_of_row(2 tq) at v_off, the next row of the fragment 128 bytes on with bit 4 of the
      // swizzled chunk turned, and the same two 8 keys further.
      const int key_a = key_of_row<D>(gid);
      // this head's first staged row, and the bytes from a key's row to that of the key 8 further: in
      // pages of 8 keys a block's halves lie behind one another with every head's 8 rows in each
      const int row0 = hl * (P8 ? 8 : kKB);
      const uint32_t next8 = (uint32_t)(8 * D * (P8 ? HB : 1));
      const uint32_t k_off = D == 128 ? row_chunk<D>(row0 + key_a, 2 * tq)
                                      : row_chunk<D>(row0 + key_a, tq);
      const uint32_t v_off =
          box_bytes + (D == 128 ? row_chunk<D>(row0 + key_of_row<D>(2 * tq), gid)
                                : row_chunk<D>(row0 + key_of_row<D>(2 * tq), gid >> 1) + (gid & 1) * 8);
      // this warp's query fragments: a lane's 8 bytes of each step, column block and fp16 part
      const uint32_t q_at = smem_u32(qfrags) + warp * q_frag_bytes(D, NB, F32) + lane * 8;
      int i0 = 0;                // block index of the piece's first block
      int s = kw, round = 0;     // stage and round of this warp's next block (kw, kw + KW, ...)
      for (int k = 0;; ++k) {
        if (!mbar_wait_warp_or_abort(&sm.pfull[k % kQueue], (uint32_t)(k / kQueue) & 1, &sm.abort_flag)) {
          give_up();
          return;
        }
        // The piece stays in its queue slot until this warp is done with it: its fields are read
        // from shared memory where they are used, not held in registers across the key loop.
        const volatile Q8Piece& d = sm.piece[k % kQueue];
        if (d.t0 < 0) break;
        auto release_piece = [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.pempty[k % kQueue]);
        };

        // ---- the request's new row of this head, quantised by the warp that will read its block:
        // lane l has values 4 l .. 4 l + 3 of K and of V (D 64: lanes 0 - 15 those of K, lanes
        // 16 - 31 those of V)
        const bool own_new = p.k_new != nullptr && d.last && (i0 + d.n - 1) % KW == kw;
        if (own_new) {
          const int t0 = d.t0, pos = d.pos0, BS = p.a.block_size;
          long long slot = __ldg(p.slot_mapping + t0);
          const int page = __ldg(p.a.block_table + (long long)d.r * p.a.bt_stride + pos / BS);
          const long long at = ((long long)t0 * Hkv + head) * D + lane * 4 % D;
          const int w = lane % (D / 4);
          float x[4];
          load4<F32>(D == 128 || lane < 16 ? p.k_new : p.v_new, at, x);
          uint32_t a = magnitude4(x);
          Q8NewRow& f = sm.fresh[warp];
          if constexpr (D == 128) {
            float y[4];
            load4<F32>(p.v_new, at, y);
            uint32_t c = magnitude4(y);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
              a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
              c = max(c, __shfl_xor_sync(0xffffffffu, c, off));
            }
            const int kc = e8m0_of_magnitude(a), vc = e8m0_of_magnitude(c);
            f.k[w] = quantise4(x, e8m0_inverse(kc));
            f.v[w] = quantise4(y, e8m0_inverse(vc));
            if (lane == 0) {
              f.k_code = kc;
              f.v_code = vc;
            }
          } else {
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
            const int code = e8m0_of_magnitude(a);
            (lane < 16 ? f.k : f.v)[w] = quantise4(x, e8m0_inverse(code));
            if (lane == 0) f.k_code = code;
            if (lane == 16) f.v_code = code;
          }
          if (slot >= (long long)p.a.num_blocks * BS) {
            if (lane == 0) record_error(p.a.error_word, CB_DEVERR_SLOT);
            slot = -1;
          }
          if (lane == 0) {
            f.row = slot < 0 ? -1 : slot * Hkv + head;
            f.staged = slot == (long long)page * BS + pos % BS;
          }
          __syncwarp();
        }

        // ---- q: column 8 nb + gid, d = D/4 tq .. + D/4 - 1, as fp16 fragments
        float cs0[NB], cs1[NB];  // score factors of columns 8 nb + 2 tq, + 1
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int col = col0 + 8 * nb + gid;
          const int tok = col >> p.lg_group;
          const bool live = tok < d.ntok;
          const long long at =
              ((long long)(d.t0 + tok) * Hq + head * G + (col & (G - 1))) * D + tq * (D / 4);
          constexpr int kRaw = F32 ? D / 4 : D / 8;  // words: fp32 values, or bf16 pairs
          uint32_t raw[kRaw];
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.a.q) + at * (F32 ? 4 : 2));
#pragma unroll
          for (int e = 0; e < kRaw / 4; ++e) {
            const uint4 v = live ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
            raw[4 * e] = v.x;
            raw[4 * e + 1] = v.y;
            raw[4 * e + 2] = v.z;
            raw[4 * e + 3] = v.w;
          }
          auto value = [&](int e) -> float {  // of d = D/4 tq + e
            if constexpr (F32) return __uint_as_float(raw[e]);
            return __uint_as_float(e & 1 ? raw[e / 2] & 0xffff0000u : raw[e / 2] << 16);
          };
          // bits of the row's largest magnitude (a row with an infinity or a NaN gives NaNs anyway)
          uint32_t top = 0u;
          if constexpr (F32) {
#pragma unroll
            for (int e = 0; e < kRaw; ++e) top = max(top, raw[e] & 0x7fffffffu);
          } else {
#pragma unroll
            for (int e = 0; e < kRaw; ++e) top = __vmaxu2(top, raw[e] & 0x7fff7fffu);
            top = max(top & 0xffff0000u, top << 16);
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = top == 0u ? 13 : max((int)(top >> 23) - 127, -100);
          const float up = __uint_as_float((uint32_t)(13 - ex + 127) << 23);
          const float cs = p.a.scale_log2 * __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
          cs0[nb] = __shfl_sync(0xffffffffu, cs, 8 * tq);
          cs1[nb] = __shfl_sync(0xffffffffu, cs, 8 * tq + 4);
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks) {
            uint32_t w[2];
            uint32_t rest[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float lo = value(4 * ks + 2 * e) * up, hi = value(4 * ks + 2 * e + 1) * up;
              w[e] = pack_f16x2(lo, hi);
              if constexpr (F32) rest[e] = pack_f16x2_rest(w[e], lo, hi);
            }
            sts64(q_at + ((ks * NB + nb) * kSplit) * 256, w[0], w[1]);
            if constexpr (F32) sts64(q_at + ((ks * NB + nb) * kSplit + 1) * 256, rest[0], rest[1]);
          }
        }
        __syncwarp();

        float o[NB][kKS][4];
        float m[NB][2], mw[NB][2], l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int e = 0; e < kKS; ++e) o[nb][e][0] = o[nb][e][1] = o[nb][e][2] = o[nb][e][3] = 0.f;
          m[nb][0] = m[nb][1] = mw[nb][0] = mw[nb][1] = kNoMax;
          l[nb][0] = l[nb][1] = 0.f;
        }
        // blocks inside this range lie inside every column's: no masks
        const int inner_lo = first_key(d.pos0 + d.ntok - 1, W), inner_hi = d.pos0;
        // this warp's blocks: global block indices congruent to kw modulo KW
        const int n = d.n, base = d.kb0 * kKB;
        for (int j = (kw - i0 % KW + KW) % KW; j < n; j += KW) {
          if (!mbar_wait_warp_or_abort(&sm.full[s], (uint32_t)round & 1, &sm.abort_flag)) {
            give_up();
            return;
          }
          const uint32_t st = stage0 + s * stage_bytes;
          const uint32_t sc = scale0 + s * 2 * scale_bytes;
          uint64_t* const done = &sm.empty[s];
          s += KW;
          if (s >= p.stages) {
            s -= p.stages;
            ++round;
          }
          const int key_base = base + j * kKB;
          const int ka = key_base + key_a, kb = ka + 8;
          if (own_new && j == n - 1) {
            const Q8NewRow& f = sm.fresh[warp];
            const int w = lane % (D / 4);
            if (f.row >= 0) {
              if (f.staged) {  // over the stale row in the staged block
                const int key = d.pos0 - key_base;
                const uint32_t at = row_chunk<D>(row0 + (key & 7), w / 4) + (key >> 3) * next8 + (w & 3) * 4;
                sts32(st + at, f.k[w]);
                sts32(st + box_bytes + at, f.v[w]);
                if (lane == 0) {
                  sts8(sc + key * Hkv, f.k_code);
                  sts8(sc + scale_bytes + key * Hkv, f.v_code);
                }
                // the producer's next copies into this stage come after these stores
                fence_proxy_async_smem();
              }
              *reinterpret_cast<uint32_t*>(p.c.k + f.row * D + w * 4) = f.k[w];
              *reinterpret_cast<uint32_t*>(p.c.v + f.row * D + w * 4) = f.v[w];
              if (lane == 0) {
                p.c.k_scale[f.row] = (uint8_t)f.k_code;
                p.c.v_scale[f.row] = (uint8_t)f.v_code;
              }
            }
            __syncwarp();
          }
          // ---- S^T = K Q^T
          // (in two chains, even and odd steps: half the dependent latency; fp32 queries keep
          // their low parts in a third, where the truncation of the large sums does not reach them)
          constexpr int kChains = F32 ? 3 : 2;
          float sc_[kChains][NB][4];
#pragma unroll
          for (int c = 0; c < kChains; ++c)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) sc_[c][nb][0] = sc_[c][nb][1] = sc_[c][nb][2] = sc_[c][nb][3] = 0.f;
#pragma unroll
          for (int half = 0; half < D / 64; ++half) {
            const uint4 va = lds128(st + (k_off ^ (half << 4)));
            const uint4 vb = lds128(st + (k_off ^ (half << 4)) + next8);
            const uint32_t wa[4] = {va.x, va.y, va.z, va.w};
            const uint32_t wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a[4] = {f16x2_lo(wa[e]), f16x2_lo(wb[e]), f16x2_hi(wa[e]), f16x2_hi(wb[e])};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const uint32_t at = q_at + (((4 * half + e) * NB + nb) * kSplit) * 256;
                const uint2 q = lds64(at);
                mma_f16_16816(sc_[e & 1][nb], a, q.x, q.y);
                if constexpr (F32) {
                  const uint2 rest = lds64(at + 256);
                  mma_f16_16816(sc_[2][nb], a, rest.x, rest.y);
                }
              }
            }
          }
          float sa[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sa[nb][e] = sc_[0][nb][e] + sc_[1][nb][e];
              if constexpr (F32) sa[nb][e] += sc_[2][nb][e];
            }
          // ---- scales: 2^ek on the score, ev in the weight's exponent
          // (scale bytes 1 .. 254: the exponent field of a normal float)
          const float fa = __uint_as_float((uint32_t)lds_u8(sc + key_a * Hkv) << 23);
          const float fb = __uint_as_float((uint32_t)lds_u8(sc + (key_a + 8) * Hkv) << 23);
          const float ea = (float)(lds_u8(sc + scale_bytes + key_a * Hkv) - kE8m0Bias);
          const float eb = (float)(lds_u8(sc + scale_bytes + (key_a + 8) * Hkv) - kE8m0Bias);
          const bool edge = key_base < inner_lo || key_base + kKB - 1 > inner_hi;  // warp-uniform
          uint32_t pw[NB][2 * kSplit];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float s0 = sa[nb][0] * cs0[nb] * fa, s1 = sa[nb][1] * cs1[nb] * fa;
            float s2 = sa[nb][2] * cs0[nb] * fb, s3 = sa[nb][3] * cs1[nb] * fb;
            float t0 = s0 + ea, t1 = s1 + ea, t2 = s2 + eb, t3 = s3 + eb;
            if (edge) {  // both: a slot that is not attended may hold any scale
              const int h0 = d.pos0 + ((col0 + 8 * nb + 2 * tq) >> p.lg_group);
              const int h1 = d.pos0 + ((col0 + 8 * nb + 2 * tq + 1) >> p.lg_group);
              const int l0 = first_key(h0, W), l1 = first_key(h1, W);
              if (ka < l0 || ka > h0) s0 = t0 = -INFINITY;
              if (ka < l1 || ka > h1) s1 = t1 = -INFINITY;
              if (kb < l0 || kb > h0) s2 = t2 = -INFINITY;
              if (kb < l1 || kb > h1) s3 = t3 = -INFINITY;
            }
            float x0 = fmaxf(s0, s2), x1 = fmaxf(s1, s3);
            float y0 = fmaxf(t0, t2), y1 = fmaxf(t1, t3);
            if (__any_sync(0xffffffffu, x0 > m[nb][0] + kRaise || x1 > m[nb][1] + kRaise ||
                                            y0 > mw[nb][0] + kRaise || y1 > mw[nb][1] + kRaise)) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
                y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, off));
                y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, off));
              }
              x0 = fmaxf(x0, m[nb][0]);
              x1 = fmaxf(x1, m[nb][1]);
              y0 = fmaxf(y0, mw[nb][0]);
              y1 = fmaxf(y1, mw[nb][1]);
              l[nb][0] *= ex2_approx(m[nb][0] - x0);
              l[nb][1] *= ex2_approx(m[nb][1] - x1);
              const float a0 = ex2_approx(mw[nb][0] - y0), a1 = ex2_approx(mw[nb][1] - y1);
              m[nb][0] = x0;
              m[nb][1] = x1;
              mw[nb][0] = y0;
              mw[nb][1] = y1;
#pragma unroll
              for (int e = 0; e < kKS; ++e) {
                o[nb][e][0] *= a0;
                o[nb][e][1] *= a1;
                o[nb][e][2] *= a0;
                o[nb][e][3] *= a1;
              }
            }
            l[nb][0] += ex2_approx(s0 - m[nb][0]) + ex2_approx(s2 - m[nb][0]);
            l[nb][1] += ex2_approx(s1 - m[nb][1]) + ex2_approx(s3 - m[nb][1]);
            const float w0 = ex2_approx(t0 - mw[nb][0] + kWeightLog2);
            const float w1 = ex2_approx(t1 - mw[nb][1] + kWeightLog2);
            const float w2 = ex2_approx(t2 - mw[nb][0] + kWeightLog2);
            const float w3 = ex2_approx(t3 - mw[nb][1] + kWeightLog2);
            const uint32_t pa = pack_f16x2(w0, w1), pb = pack_f16x2(w2, w3);
            pw[nb][0] = movmatrix_trans(pa);
            pw[nb][1] = movmatrix_trans(pb);
            if constexpr (F32) {
              pw[nb][2] = movmatrix_trans(pack_f16x2_rest(pa, w0, w1));
              pw[nb][3] = movmatrix_trans(pack_f16x2_rest(pb, w2, w3));
            }
          }
          // ---- O^T += V^T P^T
          uint32_t v[4][D / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (D == 128) {
              const uint4 x = lds128(st + (v_off ^ ((r & 1) << 4)) + (r & 1) * 128 + (r >> 1) * next8);
              v[r][0] = x.x;
              v[r][1] = x.y;
              v[r][2] = x.z;
              v[r][3] = x.w;
            } else {
              const uint2 x = lds64(st + (v_off ^ ((r & 1) << 4)) + (r & 1) * 128 + (r >> 1) * next8);
              v[r][0] = x.x;
              v[r][1] = x.y;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(done);
          if (edge) {
            // slots no row of the item attends hold anything, NaN codes too: weight 0 x value 0
            const int lo = first_key(d.pos0, W), hi = d.pos0 + d.ntok - 1;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = key_base + key_of_row<D>(2 * tq + (r & 1)) + (r >> 1) * 8;
              if (key < lo || key > hi)
#pragma unroll
                for (int e = 0; e < D / 32; ++e) v[r][e] = 0u;
            }
          }
          if (edge && d.ntok > 1) {
            // A NaN value reaches only the rows that attend its key: it is taken out of the product
            // (weight 0 x NaN), and the outputs of the rows that do attend it are set by a product
            // of indicators.
            uint32_t any = 0u;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int e = 0; e < D / 32; ++e) any |= nan_bytes(v[r][e]);
            if (__any_sync(0xffffffffu, any != 0u)) {
              uint32_t at[NB][2];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const int h0 = d.pos0 + ((col0 + 8 * nb + 2 * tq) >> p.lg_group);
                const int h1 = d.pos0 + ((col0 + 8 * nb + 2 * tq + 1) >> p.lg_group);
                const int l0 = first_key(h0, W), l1 = first_key(h1, W);
                const float a0 = ka >= l0 && ka <= h0 ? 1.f : 0.f, a1 = ka >= l1 && ka <= h1 ? 1.f : 0.f;
                const float b0 = kb >= l0 && kb <= h0 ? 1.f : 0.f, b1 = kb >= l1 && kb <= h1 ? 1.f : 0.f;
                at[nb][0] = movmatrix_trans(pack_f16x2(a0, a1));
                at[nb][1] = movmatrix_trans(pack_f16x2(b0, b1));
              }
#pragma unroll
              for (int e = 0; e < D / 32; ++e)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                  constexpr uint32_t kOne = 0x38383838u;  // 1.0 in e4m3
                  uint32_t a[4];
                  v_fragment(a, nan_bytes(v[0][e]) & kOne, nan_bytes(v[1][e]) & kOne,
                             nan_bytes(v[2][e]) & kOne, nan_bytes(v[3][e]) & kOne, hi);
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    float hit[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16_16816(hit, a, at[nb][0], at[nb][1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                      if (hit[c] > 0.f) o[nb][2 * e + hi][c] = __uint_as_float(0x7fc00000u);
                  }
                }
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < D / 32; ++e) v[r][e] &= ~nan_bytes(v[r][e]);
            }
          }
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              uint32_t a[4];
              v_fragment(a, v[0][e], v[1][e], v[2][e], v[3][e], hi);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                float(&acc)[4] = o[nb][2 * e + hi];
                if constexpr (F32) {
                  // the block's sum by itself, then added rounded to nearest: the tensor cores
                  // truncate, which over a long context would add up to a bias
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16_16816(t, a, pw[nb][2], pw[nb][3]);
                  mma_f16_16816(t, a, pw[nb][0], pw[nb][1]);
#pragma unroll
                  for (int c = 0; c < 4; ++c) acc[c] += t[c];
                } else {
                  mma_f16_16816(acc, a, pw[nb][0], pw[nb][1]);
                }
              }
            }
          }
        }
        i0 += n;

        // ---- the end of the piece: sums over the key rows of the columns
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], off);
        // ---- write: column 8 nb + 2 tq + c, outputs d = D/8 gid .. + D/8 - 1 of this lane
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = col0 + 8 * nb + 2 * tq + c;
            const int tok = col >> p.lg_group;
            if (tok >= d.ntok) continue;
            const int h = head * G + (col & (G - 1));
            // weights were relative to 2^(mw - kWeightLog2), the sum to 2^m
            float f = ex2_approx(mw[nb][c] - kWeightLog2 - m[nb][c]);
            if (d.direct) {
              f = l[nb][c] != 0.f ? f / l[nb][c] : 0.f;
              const long long at = ((long long)(d.t0 + tok) * Hq + h) * D + gid * (D / 8);
              if constexpr (F32) {
                float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at);
#pragma unroll
                for (int e = 0; e < kKS; e += 2)
                  out[e / 2] = make_float4(o[nb][e][c] * f, o[nb][e][2 + c] * f, o[nb][e + 1][c] * f,
                                           o[nb][e + 1][2 + c] * f);
              } else {
                uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + at);
#pragma unroll
                for (int e = 0; e < kKS; e += 4) {
                  uint32_t w[4];
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    w[z] = pack_bf16x2(o[nb][e + z][c] * f, o[nb][e + z][2 + c] * f);
                  out[e / 4] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            } else {
              const long long row = (((long long)d.slot * KW + kw) * TT + tok) * Hq + h;
              float4* out = reinterpret_cast<float4*>(p.part_o + row * D + gid * (D / 8));
#pragma unroll
              for (int e = 0; e < kKS; e += 2)
                out[e / 2] = make_float4(o[nb][e][c] * f, o[nb][e][2 + c] * f, o[nb][e + 1][c] * f,
                                         o[nb][e + 1][2 + c] * f);
              if (gid == 0) p.part_ml[row] = make_float2(m[nb][c], l[nb][c]);
            }
          }
        }
        release_piece();
      }
    };
    consume();
  }
  // As in the bf16 decode kernel: after a wait that gave up, the latest copy of each stage may
  // be in flight; it is waited for before the shared memory is released.
  __syncthreads();
  // (Each producer waits for its own blocks among the latest of every stage that it knows of.)
  if (producer >= 0 && lane == 0 && *reinterpret_cast<volatile int*>(&sm.abort_flag)) {
    for (int j = issued_blocks - 1; j >= 0 && j >= issued_blocks - p.stages; --j)
      if ((j / GB & (kQ8Producers - 1)) == producer)
        mbar_wait(&sm.full[j % p.stages], (uint32_t)(j / p.stages) & 1);
  }
}

// ------------------------------------------------------------------ portable kernel
//
// One CTA per (query row, KV head), for block sizes below 8 (a key block of the split kernel lies in
// one page or two), odd KV head counts in pages of 8, and more KV heads than its ring's scales
// allow. Its warps take the row's positions a few at a time in turn, each with a running (max, sum,
// output) in fp32 per query head of the group, and join through shared memory at the end. Bound by the instructions of its shuffles and
// exponentials on the row's SM: one request of 4000 positions in pages of 4, 32/8 heads, takes 174 us
// (2443 with one warp and one position in flight), 64 of 128 .. 2048 positions 295.

// Warps of a CTA, and positions a warp has in flight: as many as the group's queries and outputs
// leave registers for.
constexpr int portable_warps(int G) { return G <= 4 ? 16 : 8; }
constexpr int portable_keys(int G) { return G <= 4 ? 8 : 4; }

template <typename T, int VPT, int G>
__global__ void __launch_bounds__(portable_warps(G) * 32) q8_portable_kernel(StepArgs a, Q8Cache c) {
  constexpr int kPortableWarps = portable_warps(G), kPortableKeys = portable_keys(G);
  constexpr int D = VPT * 32;
  __shared__ float sh_o[kPortableWarps][D];
  __shared__ float2 sh_ml[kPortableWarps];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hkv = a.num_kv_heads;
  const int t = (int)(blockIdx.x / Hkv);
  const int g = (int)(blockIdx.x % Hkv);
  int lo_r = 0, hi_r = a.num_requests;
  while (hi_r - lo_r > 1) {
    const int mid = (lo_r + hi_r) >> 1;
    if (__ldg(a.query_start_loc + mid) <= t) lo_r = mid; else hi_r = mid;
  }
  const int r = lo_r;
  const int q_start = __ldg(a.query_start_loc + r);
  const int q_len = __ldg(a.query_start_loc + r + 1) - q_start;
  const int last = __ldg(a.seq_lens + r) - q_len + (t - q_start);
  const int first = first_key(last, a.sliding_window);
  const T* q = static_cast<const T*>(a.q) + ((int64_t)t * a.num_q_heads + g * G) * D + lane * VPT;
  float qv[G][VPT], m[G], l[G], o[G][VPT];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -FLT_MAX;
    l[h] = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      qv[h][v] = Elt<T>::to_f(q[h * D + v]);
      o[h][v] = 0.f;
    }
  }
  const int32_t* bt = a.block_table + (int64_t)r * a.bt_stride;
  const int lg_block = __ffs(a.block_size) - 1;  // block sizes are powers of two
  for (int64_t p0 = (int64_t)first + warp * kPortableKeys; p0 <= last; p0 += kPortableWarps * kPortableKeys) {
    uint16_t kk[kPortableKeys][VPT / 2], xx[kPortableKeys][VPT / 2];
    int kc[kPortableKeys], vc[kPortableKeys];
    bool ok[kPortableKeys];
    int64_t row[kPortableKeys];
#pragma unroll
    for (int i = 0; i < kPortableKeys; ++i) {
      const int p = (int)min(p0 + i, (int64_t)last);
      const int blk = __ldg(bt + (p >> lg_block));
      ok[i] = blk >= 0 && blk < a.num_blocks;
      if (!ok[i] && lane == 0) record_error(a.error_word, CB_DEVERR_BLOCK_ID);
      row[i] = ok[i] ? (((int64_t)blk << lg_block) + (p & (a.block_size - 1))) * Hkv + g : 0;
    }
#pragma unroll
    for (int i = 0; i < kPortableKeys; ++i) {
      kc[i] = __ldg(c.k_scale + row[i]);
      vc[i] = __ldg(c.v_scale + row[i]);
#pragma unroll
      for (int v = 0; v < VPT / 2; ++v) {
        kk[i][v] = *reinterpret_cast<const uint16_t*>(c.k + row[i] * D + lane * VPT + 2 * v);
        xx[i][v] = *reinterpret_cast<const uint16_t*>(c.v + row[i] * D + lane * VPT + 2 * v);
      }
    }
#pragma unroll
    for (int i = 0; i < kPortableKeys; ++i) {
      if (p0 + i > last) break;
      const float sk = e8m0_value(kc[i]), sv = e8m0_value(vc[i]);
      float kv[VPT], vv[VPT];
#pragma unroll
      for (int v = 0; v < VPT / 2; ++v) {
        const float2 fk = float2_of_f16x2(f16x2_of_e4m3x2(kk[i][v])), fv = float2_of_f16x2(f16x2_of_e4m3x2(xx[i][v]));
        kv[2 * v] = ok[i] ? fk.x * sk : 0.f;  // (a page id out of range reads as zeros)
        kv[2 * v + 1] = ok[i] ? fk.y * sk : 0.f;
        vv[2 * v] = ok[i] ? fv.x * sv : 0.f;
        vv[2 * v + 1] = ok[i] ? fv.y * sv : 0.f;
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) s = fmaf(qv[h][v], kv[v], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2;
        const float mn = fmaxf(m[h], s);
        const float alpha = exp2f(m[h] - mn);
        const float pe = exp2f(s - mn);
        l[h] = l[h] * alpha + pe;
#pragma unroll
        for (int v = 0; v < VPT; ++v) o[h][v] = fmaf(o[h][v], alpha, pe * vv[v]);
        m[h] = mn;
      }
    }
  }
  T* out = static_cast<T*>(a.out) + ((int64_t)t * a.num_q_heads + g * G) * D;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    __syncthreads();  // the head before has been read
    if (lane == 0) sh_ml[warp] = make_float2(m[h], l[h]);
#pragma unroll
    for (int v = 0; v < VPT; ++v) sh_o[warp][lane * VPT + v] = o[h][v];
    __syncthreads();
    if (threadIdx.x < D) {
      float M = -FLT_MAX, L = 0.f, x = 0.f;
#pragma unroll
      for (int w = 0; w < kPortableWarps; ++w) M = fmaxf(M, sh_ml[w].x);
#pragma unroll
      for (int w = 0; w < kPortableWarps; ++w) {
        const float f = exp2f(sh_ml[w].x - M);
        L += sh_ml[w].y * f;
        x += sh_o[w][threadIdx.x] * f;
      }
      const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);  // a NaN stays one
      out[h * D + threadIdx.x] = Elt<T>::from_f(x * inv);
    }
  }
}

// ------------------------------------------------------------------ host

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// A cache as (d, key in page, head, page) bytes; the box (D, 16, HB, 1) lands as rows
// (head, key) of D bytes.
cudaError_t cache_map(CUtensorMap* map, void* cache, const StepArgs& a, int hb) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t D = (cuuint64_t)a.head_dim, H = (cuuint64_t)a.num_kv_heads;
  cuuint64_t dims[4] = {D, (cuuint64_t)a.block_size, H, (cuuint64_t)a.num_blocks};
  cuuint64_t strides[3] = {H * D, D, (cuuint64_t)a.block_size * H * D};
  cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(a.block_size < kKB ? a.block_size : kKB), (cuuint32_t)hb, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, cache, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NB, bool F32, bool P8>
cudaError_t launch_split_t(const Q8Args& p, cudaStream_t s) {
  auto kern = q8_split_kernel<D, NB, F32, P8>;
  const int warps = p.heads_per_cta * p.key_warps * p.column_warps;
  const size_t smem = q8_smem_bytes(D, p.heads_per_cta, warps, NB, F32, p.stages, p.a.num_kv_heads);
  // a stage belongs to one producer and one key warp, which see every one of its phases
  const int gb = p.group_blocks;
  if (smem > (size_t)kQ8SmemLimit || gb < 1 || gb > 32 || (gb & (gb - 1)) != 0 || p.stages > kQ8MaxStages ||
      p.stages < gb * kQ8Producers || p.stages % (gb * kQ8Producers) != 0 || p.stages % p.key_warps != 0 ||
      warps > (NB == 1 ? 16 : 8))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  static DeviceFlags attr_flags;
  std::atomic<bool>& attr_set = device_flag(attr_flags);
  if (!attr_set) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kQ8SmemLimit);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  CUtensorMap mk, mv;
  e = cache_map(&mk, p.c.k, p.a, p.heads_per_cta);
  if (e == cudaSuccess) e = cache_map(&mv, p.c.v, p.a, p.heads_per_cta);
  if (e != cudaSuccess) return e;
  return launch_pdl(kDecodeQ8, kern, dim3(p.num_ctas, p.a.num_kv_heads / p.heads_per_cta),
                    dim3((warps + kQ8Producers) * 32), smem, s,
                    mk, mv, p);
}

template <int D, bool P8>
cudaError_t launch_split_d(const Q8Args& p, int nb, cudaStream_t s) {
  if (p.a.dtype == CB_F32) {
    if (nb == 1) return launch_split_t<D, 1, true, P8>(p, s);
    if (nb == 2) return launch_split_t<D, 2, true, P8>(p, s);
  } else {
    if (nb == 1) return launch_split_t<D, 1, false, P8>(p, s);
    if (nb == 2) return launch_split_t<D, 2, false, P8>(p, s);
  }
  return cudaErrorInvalidValue;
}

template <typename T, int VPT>
cudaError_t launch_portable_t(const StepArgs& a, const Q8Cache& c, cudaStream_t s) {
  const int64_t ctas = (int64_t)a.num_tokens * a.num_kv_heads;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas), block(portable_warps(a.num_q_heads / a.num_kv_heads) * 32);
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_pdl(kPortableQ8, q8_portable_kernel<T, VPT, 1>, grid, block, 0, s, a, c);
    case 2: return launch_pdl(kPortableQ8, q8_portable_kernel<T, VPT, 2>, grid, block, 0, s, a, c);
    case 4: return launch_pdl(kPortableQ8, q8_portable_kernel<T, VPT, 4>, grid, block, 0, s, a, c);
    case 8: return launch_pdl(kPortableQ8, q8_portable_kernel<T, VPT, 8>, grid, block, 0, s, a, c);
    case 16: return launch_pdl(kPortableQ8, q8_portable_kernel<T, VPT, 16>, grid, block, 0, s, a, c);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t q8_smem_bytes(int D, int HB, int warps, int NB, bool f32, int stages, int Hkv) {
  return 1024 /* alignment slack */ + (size_t)stages * (2 * HB * kKB * D + 2 * kKB * Hkv) +
         (size_t)warps * q_frag_bytes(D, NB, f32) + sizeof(Q8Smem);
}

cudaError_t launch_q8_split(const Q8Args& p, int column_blocks, cudaStream_t stream) {
  if (p.a.block_size == 8)
    return p.a.head_dim == 64 ? launch_split_d<64, true>(p, column_blocks, stream)
                              : launch_split_d<128, true>(p, column_blocks, stream);
  return p.a.head_dim == 64 ? launch_split_d<64, false>(p, column_blocks, stream)
                            : launch_split_d<128, false>(p, column_blocks, stream);
}

cudaError_t launch_q8_portable(const StepArgs& a, const Q8Cache& c, cudaStream_t stream) {
  if (a.num_tokens <= 0) return cudaSuccess;
  if (a.head_dim == 64)
    return a.dtype == CB_F32 ? launch_portable_t<float, 2>(a, c, stream)
                             : launch_portable_t<__nv_bfloat16, 2>(a, c, stream);
  return a.dtype == CB_F32 ? launch_portable_t<float, 4>(a, c, stream)
                           : launch_portable_t<__nv_bfloat16, 4>(a, c, stream);
}

}  // namespace cb
