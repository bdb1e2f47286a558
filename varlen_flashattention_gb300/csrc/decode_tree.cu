// Attention of a sequence's newest tokens, drafts of a tree or a plain chain,
// over its paged bf16 cache (jfa_decode_tree).
//
// Rows are (node i, head of the group) pairs of one KV head; row (i, g) sees
// every token t < C = L - n before the drafts and draft j iff bit j of mask_i:
//   S = scale q K^T, P = softmax(S) over the visible, O = P V, LSE = ln sum exp S.
//
// A K and a V row of one KV head serve all rows of that head: 4 D bytes for
// 4 D flops a row, so 64 rows are 64 flop per byte and 256 rows 256, against
// 288 at which the tensor cores and HBM take the same time. Below that the
// cache is read once at HBM's rate whatever the number of rows; the products
// run on tcgen05 with the rows as M = 128.
//
// A CTA holds up to two tiles of 128 rows (a row group) and works as two
// streams, each with its own score tile and accumulator in TMEM and its own
// four softmax warps. With two row tiles a stream is a row tile and both read
// every K / V tile; with one they take the K / V tiles in turn and are joined
// at the end like two parts. So one stream's softmax runs while the other's
// products do, and no stream ever waits for the other's maxima.
//
// All (sequence, KV head, row group) lines of 128-token tiles form one long
// line, which is cut evenly into one range per CTA; a line that was cut leaves
// partial results (normalised O, LSE) that a second kernel joins.
//
// Tiles are gathered through the page table: by TMA in boxes of as many tokens as
// lie side by side (the largest power of two that divides the page size); for
// pages that 8 does not divide row by row with cp.async, whose copies arrive at the
// tile's barrier themselves (95% of the copy rate; waited for by their warp before it
// announced the tile, and looked up one by one, 72%; TMA's gather of four rows, 56%).
// Drafts are the last tokens, so only a line's last one or two tiles have a
// mask. In those V rows that some row may not see are checked first: what is
// not finite there becomes 0 for the product, since 0 * NaN would reach every
// row, and is added to the rows that do see it at the end. Where partial results are joined a weight that has
// underflowed to 0 still multiplies, so that NaN and infinities are kept wherever the line was cut.
//
// Roles (384 threads): warps 0-3 and 4-7 the streams' softmax and epilogue, warp
// 8 K loads, warp 9 Q and V loads, warp 10 MMA issuer, warp 11 the scheduler,
// which walks the CTA's range and hands its items to the others through a ring in
// shared memory. (With a walk in each role, the code that only item borders run came
// from DRAM again and again, past the stream of K and V in L2: an item cost 7.7 us.)
//
// Measured, 8 KV heads of 128, pages of 16, device time with the join: 32 x 1k-32k tokens,
// 4 rows a head 328-339 us by the card (98-100% of the copy rate), 64 rows 338-348 (96-98%), 256
// rows 406-427 (79-83%). Where rows are many the chain of one stream is the bound (softmax 1860
// cycles, then its products behind the other stream's, 1024 each, and barriers between): 16 x
// 0.5k-8k with 512 rows on 4 heads 74 us, tensor cores busy 46% of the cycles. Where lines are
// short it is the chain at a line's end: 512 x 1-300 tokens 144-147 us, 33% of the copy rate.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8_cache.cuh"  // FastDiv
#include "jfa_internal.h"
#include "ptx.cuh"

namespace jfa {

namespace {

constexpr int kTreeThreads = 384;
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpWalk = 11;
constexpr int kItemRing = 4;        // items handed out ahead
constexpr int kItemConsumers = 11;  // every warp but the scheduler
constexpr float kLn2f = 0.6931471805599453f;

struct TreeParams {
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* q_offsets;
  const uint64_t* mask;  // may be null: a chain
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  __nv_bfloat16* o;
  float* lse;
  TreeBuffers w;
  int32_t batch, hq, hkv, group, num_pages, max_pages, total_q, max_q;
  int32_t nodes_per_tile;  // nodes whose rows fit a tile: 128 / group
  uint32_t node_tile_mul;  // 2^16 / nodes_per_tile + 1: x / nodes_per_tile = x * this >> 16 for x < 512
  FastDiv page;            // division by page_size
  int32_t box;             // tokens of a box, or 1: rows are copied one by one
  float scale_log2;
  uint64_t budget_ns;
};

template <int D>
struct TreeLayout {
  static constexpr int kTileBytes = kTile * D * 2;  // a Q, K or V tile
  // K tiles are free once S is computed, V tiles wait for the softmax: three of the five slots that fit
  static constexpr int kSlotsK = D == 128 ? 2 : 4, kSlotsV = D == 128 ? 3 : 6;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kSlotsK * kTileBytes;
  static constexpr int kOffMl = kOffV + kSlotsV * kTileBytes;   // float2 (m, l) per stream and row
  static constexpr int kOffItems = kOffMl + 2 * kTile * 8;      // int4[3] per item
  static constexpr int kOffBars = kOffItems + kItemRing * 48;
  // k_full, k_empty, v_full, v_empty, item_full, item_empty, q_full, q_empty, s_full[2], p_half[2], p_full[2],
  // o_full[2], o_free, ml_full[2], drain, scan_ask, scan_done
  static constexpr int kNumBars = 2 * kSlotsK + 2 * kSlotsV + 2 * kItemRing + 2 + 8 + 1 + 2 + 1 + 2;
  static constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kBytes = kOffMisc + 176;
  static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;  // S: 128 columns a stream, O: D
  static_assert(kBytes <= 232448, "shared memory budget");
};

// A CTA's share of one line, as the scheduler hands it out (b = -1: the end).
struct TreeItem {
  int b, h, tile0, two;  // sequence, KV head, first row tile, two row tiles
  int t0, t1, nt, L;     // tiles of the line, of how many, tokens
  int q0, n;             // first row of q, nodes
};

// The sequence's new tokens and length; false where they are out of range (reported by the numbering).
__device__ __forceinline__ bool tree_seq(const TreeParams& p, int b, int& q0, int& n, int& L) {
  q0 = p.q_offsets[b];
  const int q1 = p.q_offsets[b + 1];
  L = p.seqlens[b];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.total_q && q1 - q0 <= p.max_q && L >= q1 - q0 &&
                  L <= static_cast<int64_t>(p.num_pages ? p.max_pages : 0) * p.page.d && (b > 0 || q0 == 0);
  n = ok ? q1 - q0 : 0;
  return ok;
}
__device__ __forceinline__ int row_tiles(const TreeParams& p, int n) {
  return static_cast<int>((static_cast<uint32_t>(n + p.nodes_per_tile - 1) * p.node_tile_mul) >> 16);
}
// A line's end (its mask, the last products, the results, the next line's Q) takes about as long as this many
// tiles, so it counts like them when the work is split. (16 x 0.5k-8k tokens with 512 rows a head: 81 us if it
// counts 1, 77 for 2, 74 for 3, 78 for 4; 512 x 1-300 tokens of one row tile 138, 140, 144, 149.)
constexpr int kLineCost = 3;
// What all the sequence's lines cost, in tiles (below 2^31: the entry point sees to that).
__device__ __forceinline__ uint32_t seq_work(const TreeParams& p, int n, int L) {
  if (n == 0) return 0;
  return static_cast<uint32_t>(p.hkv) * ((row_tiles(p, n) + 1) >> 1) *
         static_cast<uint32_t>(((L + kTile - 1) >> 7) + kLineCost);
}
// Where CTA c's share of the work begins.
__device__ __forceinline__ uint32_t share_begin(uint32_t total, uint32_t ctas, uint32_t c) {
  const uint32_t each = total / ctas;
  return c * each + min(c, total - each * ctas);
}

// Walks the items of a range of the long line; a whole warp calls it.
struct TreeWalk {
  int b, h, rg, x, q0, n, L, nt, groups;  // x: where in its line, in units of cost (from nt on: behind its tiles)
  uint32_t left;
  __device__ __forceinline__ void seq(const TreeParams& p) {
    nt = (L + kTile - 1) >> 7;
    groups = (row_tiles(p, n) + 1) >> 1;
  }
  __device__ __forceinline__ void open(const TreeParams& p, int4 first, uint32_t pos, uint32_t len) {
    left = len;
    b = first.x;
    q0 = first.y;
    n = first.z;
    L = first.w;
    seq(p);
    const uint32_t each = static_cast<uint32_t>(nt + kLineCost), line = pos / each;
    x = static_cast<int>(pos - line * each);
    h = static_cast<int>(line / static_cast<uint32_t>(groups));
    rg = static_cast<int>(line) - h * groups;
  }
  __device__ __forceinline__ void next_line(const TreeParams& p) {
    x = 0;
    if (left == 0 || ++rg < groups) return;
    rg = 0;
    if (++h < p.hkv) return;
    h = 0;
    // the next sequence with new tokens, 32 looked at together (there is one: work is left)
    for (int from = b + 1; from < p.batch; from += 32) {
      const int at = from + static_cast<int>(threadIdx.x & 31);
      int aq = 0, an = 0, al = 0;
      const bool some = at < p.batch && tree_seq(p, at, aq, an, al) && an > 0;
      const uint32_t m = __ballot_sync(0xffffffffu, some);
      if (m) {
        const int src = __ffs(m) - 1;
        b = from + src;
        q0 = __shfl_sync(0xffffffffu, aq, src);
        n = __shfl_sync(0xffffffffu, an, src);
        L = __shfl_sync(0xffffffffu, al, src);
        seq(p);
        return;
      }
    }
    left = 0;  // only if the arrays changed under the call
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeItem& I) {
    if (left > 0 && x >= nt) {
      left -= min(left, static_cast<uint32_t>(nt + kLineCost - x));
      next_line(p);
    }
    if (left == 0) return false;
    I.b = b;
    I.h = h;
    I.tile0 = 2 * rg;
    I.two = row_tiles(p, n) - 2 * rg >= 2;
    I.t0 = x;
    I.t1 = x + static_cast<int>(min(static_cast<uint32_t>(nt - x), left));
    I.nt = nt;
    I.L = L;
    I.q0 = q0;
    I.n = n;
    left -= I.t1 - I.t0;
    x = I.t1;
    return true;
  }
};

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          ptx::smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// 16 bytes from global to shared memory, part of the thread's copy group.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives at the barrier once the thread's copies so far have been written.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// acc + 0 * v in the halves: NaN from then on once a value is infinite or NaN.
__device__ __forceinline__ __nv_bfloat162 not_finite(__nv_bfloat162 acc, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(w + i), __nv_bfloat162(0.f, 0.f), acc);
  return acc;
}
// The values of a word that are finite, 0 for the others.
__device__ __forceinline__ uint32_t keep_finite(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

// Adds the non-finite values of the flagged drafts that a row sees to columns c .. end of what it has
// written: its row of O, or its partial result (rare: kept out of line, and off the registers of the
// item's end).
__device__ __noinline__ void add_not_finite(const TreeParams& p, int b, int kv_row, int first, uint64_t flags, int D,
                                            int c, int end, __nv_bfloat16* whole, float* part) {
  while (flags) {
    const int t = first + __ffsll(static_cast<long long>(flags)) - 1;
    flags &= flags - 1;
    const int pg = fast_div(t, p.page), slot = t - pg * static_cast<int>(p.page.d);
    const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pg];
    const int64_t row =
        static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages) ? static_cast<int64_t>(page) * p.page.d + slot : slot;
    const __nv_bfloat16* v = p.v_cache + (row * p.hkv + kv_row) * D;
#pragma unroll 1
    for (int e = c; e < end; ++e) {
      const float x = __bfloat162float(v[e]);
      if (fabsf(x) < INFINITY) continue;
      if (whole)
        whole[e] = __float2bfloat16(__bfloat162float(whole[e]) + x);
      else
        part[(e / 4) * 4 * kTile + e % 4] += x;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using Lay = TreeLayout<D>;
  constexpr int kSlotsK = Lay::kSlotsK, kSlotsV = Lay::kSlotsV;
  constexpr int kAtoms = D / 64;  // 64-column atoms of a tile
  constexpr int kHalf = D / 2;
  constexpr uint32_t kIdS = ptx::idesc_bf16(kTile, kTile, false, false);  // S = Q K^T
  constexpr uint32_t kIdPV = ptx::idesc_bf16(kTile, D, false, true);      // O += P V, P from TMEM

  extern __shared__ uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBars);
  uint64_t* k_empty = k_full + kSlotsK;
  uint64_t* v_full = k_empty + kSlotsK;
  uint64_t* v_empty = v_full + kSlotsV;
  uint64_t* item_full = v_empty + kSlotsV;
  uint64_t* item_empty = item_full + kItemRing;
  uint64_t* q_full = item_empty + kItemRing;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* p_half = s_full + 2;  // P of keys 64-127, which the products start with
  uint64_t* p_full = p_half + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* ml_full = o_free + 1;
  uint64_t* drain = ml_full + 2;
  uint64_t* scan_ask = drain + 1;  // V of a tile with drafts has arrived / has been looked over
  uint64_t* scan_done = drain + 2;
  float2* ml = reinterpret_cast<float2*>(smem + Lay::kOffMl);
  int4* items = reinterpret_cast<int4*>(smem + Lay::kOffItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::kOffMisc);
  ptx::CtaCtl* ctl = reinterpret_cast<ptx::CtaCtl*>(smem + Lay::kOffMisc + 8);
  // the sequence in which the range begins (its number, first row, nodes, tokens), and where in its lines
  int4* s_first = reinterpret_cast<int4*>(smem + Lay::kOffMisc + 160);
  uint32_t* s_pos = reinterpret_cast<uint32_t*>(smem + Lay::kOffMisc + 20);
  unsigned long long* s_flags = reinterpret_cast<unsigned long long*>(smem + Lay::kOffMisc + 32);  // [4]
  int2* scan_slot = reinterpret_cast<int2*>(smem + Lay::kOffMisc + 24);  // what scan_ask asks for
  unsigned long long* s_sum = reinterpret_cast<unsigned long long*>(smem + Lay::kOffMisc + 64);    // [kTreeThreads / 32]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  int32_t* status = p.w.cta_status + 2 * cta;
  allow_next_grid();
  if ((ptx::smem_u32(smem) & 1023) != 0) {  // not aligned enough for the layout
    if (tid == 0) {
      status[0] = JFA_ERR_UNSUPPORTED;
      status[1] = 0;
      if (cta == 0) *p.w.total = 0;
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kSlotsK; ++i) {
      ptx::mbar_init(k_full + i, p.box > 1 ? 1 : 32);  // row by row every lane arrives
      ptx::mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < kSlotsV; ++i) {
      ptx::mbar_init(v_full + i, p.box > 1 ? 1 : 32);
      ptx::mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < kItemRing; ++i) {
      ptx::mbar_init(item_full + i, 1);
      ptx::mbar_init(item_empty + i, kItemConsumers);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_full + i, 1);
      ptx::mbar_init(p_half + i, 4);  // the stream's softmax warps
      ptx::mbar_init(p_full + i, 4);
      ptx::mbar_init(o_full + i, 1);
      ptx::mbar_init(ml_full + i, 4);
    }
    ptx::mbar_init(o_free, 8);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(scan_ask, 1);
    ptx::mbar_init(scan_done, 1);
    for (int i = 0; i < 4; ++i) s_flags[i] = 0;
    ctl->abort = 0;
    status[0] = 0;
    status[1] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kWarpK && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  if (warp == kWarpMma) {
    ptx::tmem_alloc(tmem_slot, Lay::kTmemCols);
    ptx::tmem_relinquish();
  }
  __syncthreads();  // the status words are cleared

  // ---------------------------------------------------------------- numbering
  // The work of all lines is summed, then the sequence in which this CTA's range begins is found.
  unsigned long long sum = 0;
  int q0 = 0, n = 0, L = 0;  // the sequence that this thread numbers (its only one in batches up to the block)
  // Reports the input; the rows of q from first_row to end_row are empty, a share of them a CTA.
  auto refuse = [&](int first_row, int end_row) {
    atomicCAS(status, JFA_OK, JFA_ERR_BAD_INPUT);
    atomicCAS(status + 1, 0, kSiteTreeInput);
    const int64_t to = static_cast<int64_t>(min(end_row, p.total_q)) * p.hq;
    for (int64_t i = static_cast<int64_t>(max(first_row, 0)) * p.hq + cta; i < to; i += gridDim.x) {
      p.lse[i] = -INFINITY;
      for (int c = 0; c < D; c += 8) ptx::st_v4(p.o + i * D + c, 0, 0, 0, 0);
    }
  };
  {
    unsigned long long mine = 0;
    for (int b = tid; b < p.batch; b += kTreeThreads) {
      if (!tree_seq(p, b, q0, n, L)) refuse(q0, p.q_offsets[b + 1]);
      mine += seq_work(p, n, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTreeThreads / 32; ++i) sum += s_sum[i];
  }
  // The work is numbered with 31 bits; 2^31 tiles would take this kernel some twenty seconds (1.5 us a tile of 128 x
  // 128 at the copy rate, 152 at a time). Lines that share pages can come to more: no sequence is done then.
  if (sum >= (1ull << 31)) {
    for (int b = tid; b < p.batch; b += kTreeThreads) refuse(p.q_offsets[b], p.q_offsets[b + 1]);
    sum = 0;
  }
  // one range a CTA; with fewer tiles than CTAs the last ones have none
  const uint32_t total = static_cast<uint32_t>(sum), ctas = min(gridDim.x, total);
  const uint32_t begin = static_cast<uint32_t>(cta) < ctas ? share_begin(total, ctas, cta) : 0;
  const uint32_t end = static_cast<uint32_t>(cta) < ctas ? share_begin(total, ctas, cta + 1) : 0;
  if (cta == 0 && tid == 0) *p.w.total = total;
  if (begin < end) {
    uint32_t base = 0;
    for (int b0 = 0; b0 < p.batch && base <= begin; b0 += kTreeThreads) {
      if (p.batch > kTreeThreads) {
        n = 0;
        if (b0 + tid < p.batch) tree_seq(p, b0 + tid, q0, n, L);
      }
      const uint32_t v = seq_work(p, n, L);
      uint32_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int i = 0; i < kTreeThreads / 32; ++i) {
        if (i == warp) incl += base + all;
        all += static_cast<uint32_t>(s_sum[i]);
      }
      if (begin < incl && begin >= incl - v) {
        *s_first = make_int4(b0 + tid, q0, n, L);
        *s_pos = begin - (incl - v);
      }
      base += all;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t budget = p.budget_ns;
  TreeItem I{};
  // The next item: entry k of the ring. False at the end, or when a wait gave up.
  auto take = [&](uint32_t k) -> bool {
    const uint32_t e = k % kItemRing;
    if (!ptx::warp_all(ptx::mbar_wait(item_full + e, (k / kItemRing) & 1, ctl, status, kSiteTreeItem, budget)))
      return false;
    const int4 a = items[3 * e], c = items[3 * e + 1], d = items[3 * e + 2];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(item_empty + e);
    I = TreeItem{a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w, d.x, d.y};
    return I.b >= 0;
  };

  if (warp == kWarpWalk) {
    // ------------------------------------------------------------ scheduler
    TreeWalk walk{};
    if (begin < end) {
      walk.open(p, *s_first, *s_pos, end - begin);
      if (lane == 0) {  // where this CTA's range begins, for the join (behind a line's tiles: at the next line)
        p.w.records[2 * cta] = make_int4(walk.b, walk.h, walk.rg, walk.x < walk.nt ? walk.x : 0);
        p.w.records[2 * cta + 1] = make_int4(walk.nt, walk.q0, walk.n, row_tiles(p, walk.n) - 2 * walk.rg >= 2);
      }
    }
    // Two things to do in the order they come up: the next item, once the ring has an entry for it; and V of a
    // tile with drafts, which the MMA warp asks for. What is not finite there, of a draft that some row may not see or
    // behind the last token, becomes 0 for the product; drafts with such values are flagged for the item's end.
    TreeItem J{};
    bool more = true, due = true, given = false;
    uint32_t items_out = 0, scans = 0;
    while (true) {
      bool idle = true;
      if (due) {  // the walk's only copy: what runs once an item has to be small to stay in the instruction caches
        more = walk.next(p, J);
        due = idle = false;
      } else if (!given) {
        const uint32_t e = items_out % kItemRing;
        if (ptx::warp_all(ptx::mbar_test(item_empty + e, ((items_out / kItemRing) & 1) ^ 1))) {
          idle = false;
          if (lane == 0) {
            items[3 * e] = make_int4(more ? J.b : -1, J.h, J.tile0, J.two);
            items[3 * e + 1] = make_int4(J.t0, J.t1, J.nt, J.L);
            items[3 * e + 2] = make_int4(J.q0, J.n, 0, 0);
            ptx::mbar_arrive(item_full + e);  // release: the record is visible to the entry's waiters
          }
          __syncwarp();
          ++items_out;
          due = more;
          given = !more;
        }
      }
      if (ptx::warp_all(ptx::mbar_test(scan_ask, scans & 1))) {
        idle = false;
        const int2 ask = *scan_slot;  // (V slot, draft number of its first token)
        const uint32_t item = ask.x >> 8;
        uint8_t* v = smem + Lay::kOffV + (ask.x & 255) * Lay::kTileBytes;
        // half a warp a row (a quarter at D = 64); the swizzle only orders a row's chunks, so all are looked at
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAhead = 8;
        const int c = lane % kLanes;
        uint8_t* col = v + (c >> 3) * 16384 + (c & 7) * 16;
        bool dirty = false;
        for (int r0 = max(0, -ask.y) / kRows * kRows + lane / kLanes; r0 < kTile; r0 += kRows * kAhead) {
          uint4 x[kAhead];
#pragma unroll
          for (int e = 0; e < kAhead; ++e)
            x[e] = r0 + e * kRows < kTile ? *reinterpret_cast<uint4*>(col + (r0 + e * kRows) * 128) : make_uint4(0, 0, 0, 0);
          __nv_bfloat162 acc(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < kAhead; ++e) acc = not_finite(acc, x[e]);
          if (!__hisnan(acc.x) && !__hisnan(acc.y)) continue;
#pragma unroll 1
          for (int e = 0; e < kAhead; ++e) {
            const int r = r0 + e * kRows, draft = ask.y + r;
            if (r >= kTile || draft < 0) continue;
            uint32_t* w = reinterpret_cast<uint32_t*>(col + r * 128);
            bool found = false;
            for (int i = 0; i < 4; ++i) found = found || keep_finite(w[i]) != w[i];
            if (!found) continue;
            dirty = true;
            if (draft < kTreeMaxNodes) {
              atomicOr(s_flags + (item & 3), 1ull << draft);  // bits past the drafts meet no row's mask
              __threadfence_block();
            }
            for (int i = 0; i < 4; ++i) w[i] = keep_finite(w[i]);
          }
        }
        if (dirty) ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(scan_done);
        ++scans;
      }
      if (given && ptx::warp_all(ptx::mbar_test(drain, 0))) break;
      if (idle) {
        if (__any_sync(0xffffffffu, ctl->abort != 0)) break;  // whoever waits for this warp gives up in time
        __nanosleep(40);
      }
    }
  } else if (warp == kWarpK || warp == kWarpV) {
    // ------------------------------------------------------------ K loads; Q and V loads
    const bool is_v = warp == kWarpV;
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    const uint32_t slots = is_v ? kSlotsV : kSlotsK;
    uint8_t* ring = smem + (is_v ? Lay::kOffV : Lay::kOffK);
    const uint32_t q_bytes = static_cast<uint32_t>(p.nodes_per_tile * p.group) * 128 * kAtoms;
    uint32_t slot = 0, phase = 1, loads = 0, nq = 0;
    bool ok = true, bad = false;
    const int box = p.box;
    const char* cache = reinterpret_cast<const char*>(is_v ? p.v_cache : p.k_cache);
    auto copy_rows = [&](uint32_t dst, const int (&y)[4], int valid) {
      constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a step
      const int c = lane % kLanes, sub = lane / kLanes;
      const char* src = cache + (static_cast<int64_t>(I.h) * D + 8 * c) * 2;
      const int64_t row_bytes = static_cast<int64_t>(p.hkv) * D * 2;
      dst += (c >> 3) * 16384 + sub * 128;
      uint32_t swizzled[8 / kRows];  // the chunk's place in rows sub, sub + kRows, .. of eight
#pragma unroll
      for (int i = 0; i < 8 / kRows; ++i) swizzled[i] = dst + (((c & 7) ^ (i * kRows + sub)) << 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int from[32 / kRows];  // all looked up before the first copy: a shuffle's latency once
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i) from[i] = __shfl_sync(0xffffffffu, y[e], i * kRows + sub);
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i) {
          const int r = 32 * e + i * kRows;  // and sub more
          if (r + sub < valid) cp_async16(swizzled[i % (8 / kRows)] + r * 128, src + from[i] * row_bytes);
        }
      }
    };
    // The tokens of a tile whose pages this lane looks up: the first of a box (as many lanes as boxes, once
    // for each atom), or every 32nd; past the sequence's end its last token again.
    auto page_of = [&](int t) -> int {
      return p.page_table[static_cast<int64_t>(I.b) * p.max_pages + fast_div(t, p.page)];
    };
    auto row_of = [&](int t, int page) -> int {  // in the [num_pages * page_size, hkv * D] view
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
        bad = true;
        page = 0;
      }
      return page * static_cast<int>(p.page.d) + t - fast_div(t, p.page) * static_cast<int>(p.page.d);
    };
    auto token = [&](int tile, int e) -> int {
      return min(tile * kTile + (box > 1 ? (lane & 15) * box : 32 * e + lane), I.L - 1);
    };
    for (uint32_t it = 0; ok && take(it); ++it) {
      int pg[4];
      const int per = box > 1 ? 1 : 4;
      for (int e = 0; e < 4; ++e) pg[e] = e < per ? page_of(token(I.t0, e)) : 0;
      if (is_v) {
        ok = ptx::warp_all(ptx::mbar_wait(q_empty, (it & 1) ^ 1, ctl, status, kSiteTreeProdQ, budget));
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(q_full, q_bytes * (I.two ? 2 : 1));
          for (int m = 0; m <= I.two; ++m)
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
              tma_load_3d(smem + Lay::kOffQ + m * Lay::kTileBytes + a * 16384, &tm_q, q_full, 64 * a, I.h * p.group,
                          I.q0 + (I.tile0 + m) * p.nodes_per_tile);
        }
        __syncwarp();
        ++nq;
      }
      const int x = I.h * D;
      for (int t = I.t0; t < I.t1; ++t) {
        const int valid = min(kTile, I.L - t * kTile);
        int y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = e == 0 || box == 1 ? row_of(token(t, e), pg[e]) : 0;
        if (t + 1 < I.t1) {  // the next tile's pages, on their way while this one's slot is waited for
          pg[0] = page_of(token(t + 1, 0));
          if (box == 1) {
#pragma unroll
            for (int e = 1; e < 4; ++e) pg[e] = page_of(token(t + 1, e));
          }
        }
        uint8_t* dst = ring + slot * Lay::kTileBytes;
        ok = ptx::warp_all(ptx::mbar_wait(empty + slot, phase, ctl, status, kSiteTreeProdSlot, budget));
        if (!ok) break;
        if (box > 1) {
          const int pieces = (valid + box - 1) / box;
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(full + slot, static_cast<uint32_t>(pieces * box * 128 * kAtoms));
          __syncwarp();
          // at most 16 boxes: a half warp an atom
          const int i = lane & 15, a = lane >> 4;
          if (a < kAtoms && i < pieces)
            ptx::tma_load_2d(dst + a * 16384 + i * box * 128, map, full + slot, x + 64 * a, y[0]);
          __syncwarp();
        } else {
          copy_rows(ptx::smem_u32(dst), y, valid);
          cp_async_arrive(full + slot);
        }
        ++loads;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    cp_async_wait_all();
    if (__any_sync(0xffffffffu, bad) && lane == 0) {
      atomicCAS(status, JFA_OK, JFA_ERR_BAD_INPUT);
      atomicCAS(status + 1, 0, kSiteTreeInput);
    }
    // after an abort some loads may have no consumer: none may be in flight when the CTA exits
    if (lane == 0) {
      ptx::CtaCtl no_abort{0, 0};
      for (uint32_t i = loads > slots ? loads - slots : 0; box > 1 && i < loads; ++i)
        ptx::mbar_wait(full + i % slots, (i / slots) & 1, &no_abort, nullptr, kSiteTreeDrain, budget);
      if (nq > 0) ptx::mbar_wait(q_full, (nq - 1) & 1, &no_abort, nullptr, kSiteTreeDrain, budget);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop; one elected lane issues. A look at a barrier takes some 300 cycles while
    // MMAs read shared memory, so barriers are looked at ahead, and the answer is taken after the next MMAs.
    // One warp for both streams: with a warp each they fall into step, both softmaxes beside idle tensor
    // cores (one sequence of 131k tokens and 240 rows: 140 us against 118).
    uint32_t it = 0, scans = 0, np[2] = {0, 0}, kslot = 0, kphase = 0, vslot = 0, vphase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase, int site, bool ahead = false) -> bool {
      if (!ahead) ok = ptx::warp_all(ptx::mbar_wait(bar, phase, ctl, status, site, budget));
      return ok;
    };
    auto k_look = [&]() { return ptx::mbar_test(k_full + kslot, kphase); };
    auto v_look = [&]() { return ptx::mbar_test(v_full + vslot, vphase); };
    auto p_look = [&](int g) { return ptx::mbar_test(p_half + g, np[g] & 1); };
    auto k_wait = [&](bool ahead = false) -> uint32_t {
      const uint32_t slot = kslot;
      wait(k_full + slot, kphase, kSiteTreeMmaSlot, ahead);
      if (p.box == 1) ptx::fence_proxy_async_smem();  // the products read what ordinary copies have written
      if (++kslot == kSlotsK) {
        kslot = 0;
        kphase ^= 1;
      }
      return slot;
    };
    auto v_wait = [&](bool ahead = false) -> uint32_t {
      const uint32_t slot = vslot;
      wait(v_full + slot, vphase, kSiteTreeMmaSlot, ahead);
      if (p.box == 1) ptx::fence_proxy_async_smem();
      if (++vslot == kSlotsV) {
        vslot = 0;
        vphase ^= 1;
      }
      return slot;
    };
    // S of stream g over the K tile in `slot`; free_slot and free_q: its last readers
    auto issue_s = [&](int g, int qtile, uint32_t slot, bool free_slot, bool free_q) {
      const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(smem + Lay::kOffQ + qtile * Lay::kTileBytes), 16, 1024);
      const uint64_t k_desc = ptx::sdesc_sw128(ptx::smem_u32(smem + Lay::kOffK + slot * Lay::kTileBytes), 16, 1024);
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          ptx::mma_ss(tmem + Lay::kColS + g * kTile, q_desc + (off >> 4), k_desc + (off >> 4), kIdS, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(s_full + g);
        if (free_slot) ptx::mma_commit(k_empty + slot);
        if (free_q) ptx::mma_commit(q_empty);
      }
      __syncwarp();
    };
    // V of tile t has arrived: is it one with drafts?
    auto has_drafts = [&](int t) -> bool { return (I.t0 + t + 1) * kTile > I.L - I.n; };
    auto ask_scan = [&](int t, uint32_t slot) {
      if (!has_drafts(t)) return;
      if (ptx::elect_one()) {
        *scan_slot = make_int2(static_cast<int>(slot | it << 8), (I.t0 + t) * kTile - (I.L - I.n));
        ptx::mbar_arrive(scan_ask);  // release: the slot is visible to the scheduler
      }
      __syncwarp();
    };
    auto issue_pv = [&](int g, int t, uint32_t slot, bool first, bool last, bool free_slot, bool ahead) {
      if (first && it > 0 && !wait(o_free, (it - 1) & 1, kSiteTreeMmaOFree)) return;  // read out of the accumulators
      if ((g == 0 || !I.two) && has_drafts(t) && !wait(scan_done, scans++ & 1, kSiteTreeMmaScan)) return;
      if (!ahead && !wait(p_half + g, np[g] & 1, kSiteTreeMmaP)) return;
      ptx::tc_fence_after();  // P and the accumulators were last touched by the softmax warps
      const uint64_t v_desc =
          ptx::sdesc_sw128(ptx::smem_u32(smem + Lay::kOffV + slot * Lay::kTileBytes), 16384, 1024);
      const uint32_t o = tmem + Lay::kColO + g * D, pt = tmem + Lay::kColS + g * kTile + 64;
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 4; kk < 8; ++kk)
          ptx::mma_ts(o, pt + kk * 8, v_desc + ((kk * 2048) >> 4), kIdPV, (!first || kk > 4) ? 1u : 0u);
      }
      __syncwarp();
      if (!wait(p_full + g, np[g] & 1, kSiteTreeMmaP)) return;
      ++np[g];
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) ptx::mma_ts(o, pt + kk * 8, v_desc + ((kk * 2048) >> 4), kIdPV, 1u);
        if (free_slot) ptx::mma_commit(v_empty + slot);
        if (last) ptx::mma_commit(o_full + g);
      }
      __syncwarp();
    };
    while (ok && take(it)) {
      const int nt = I.t1 - I.t0;
      if (!wait(q_full, it & 1, kSiteTreeMmaQ)) break;
      uint32_t ks = k_wait();
      if (!ok) break;
      if (I.two) {
        issue_s(0, 0, ks, false, false);
        issue_s(1, 1, ks, true, nt == 1);
        uint32_t vs = v_wait();
        if (!ok) break;
        ask_scan(0, vs);
        if (nt > 1) ks = k_wait();
        for (int t = 0; ok && t < nt; ++t) {
          const bool more = t + 1 < nt;
          issue_pv(0, t, vs, t == 0, !more, false, false);
          if (!ok) break;
          const bool p1 = p_look(1);
          if (more) issue_s(0, 0, ks, false, false);
          issue_pv(1, t, vs, t == 0, !more, true, ptx::warp_all(p1));
          if (!ok) break;
          if (more) {
            const bool v = v_look();
            const uint32_t at = ks;
            const bool next = t + 2 < nt, k = next && k_look();
            issue_s(1, 1, at, true, !next);
            const bool here = ptx::warp_all(v && (k || !next));
            vs = v_wait(here);
            if (!ok) break;
            ask_scan(t + 1, vs);
            if (next) ks = k_wait(here);
          }
        }
      } else {
        issue_s(0, 0, ks, true, nt == 1);
        if (nt > 1) {
          ks = k_wait();
          if (!ok) break;
          issue_s(1, 0, ks, true, nt == 2);
        }
        bool v = false;
        for (int t = 0; ok && t < nt; ++t) {
          const bool more = t + 2 < nt;
          const uint32_t vs = v_wait(ptx::warp_all(v));
          if (!ok) break;
          ask_scan(t, vs);
          const bool k = more && k_look();
          issue_pv(t & 1, t, vs, t < 2, t + 2 >= nt, true, false);
          if (!ok) break;
          v = t + 1 < nt && v_look();
          if (more) {
            ks = k_wait(ptx::warp_all(k));
            if (!ok) break;
            issue_s(t & 1, 0, ks, true, t + 3 == nt);
          }
        }
      }
      ++it;
    }
    if (ptx::elect_one()) ptx::mma_commit(drain);
    __syncwarp();
    ptx::CtaCtl no_abort{0, 0};
    // the scheduler waits for it too, with no limit of its own but the abort flag
    if (!ptx::mbar_wait(drain, 0, &no_abort, status, kSiteTreeDrain, budget)) ctl->abort = 1;
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and epilogue (warps 0-7)
    const int g = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + Lay::kColS + g * kTile;
    const uint32_t o_tmem = tmem + lane_base + Lay::kColO;
    const int row_node = r / p.group, row_head = r % p.group;  // of this row in its tile
    const float sl = p.scale_log2;
    const uint64_t sl2 = ptx::f2_packf(sl, sl);
    uint32_t ns = 0, it = 0;
    uint32_t no0 = 0, no1 = 0, nml0 = 0, nml1 = 0;  // phases of o_full and ml_full so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase, int site) -> bool {  // the warp agrees, so that votes below are whole
      return ok = ptx::warp_all(ptx::mbar_wait(bar, phase & 1, ctl, status, site, budget));
    };
    while (ok && take(it)) {
      const int nt = I.t1 - I.t0, C = I.L - I.n;
      const int node = (I.tile0 + (I.two ? g : 0)) * p.nodes_per_tile + row_node;
      const bool row_ok = row_node < p.nodes_per_tile && node < I.n;
      const bool active = __any_sync(0xffffffffu, row_ok);
      uint64_t bits = 0;  // the drafts that this row sees
      if (row_ok) {
        bits = p.mask ? p.mask[I.q0 + node] : (~uint64_t(0) >> (63 - node));
        bits &= ~uint64_t(0) >> (64 - I.n);
      }
      if (g == 0 && tid == 0) s_flags[(it + 2) & 3] = 0;
      float m = -INFINITY, l = 0.f;
      const int step = I.two ? 1 : 2;
      for (int t = I.two ? 0 : g; t < nt; t += step) {
        const int tok = (I.t0 + t) * kTile;
        const bool masked = tok + kTile > C;
        if (!wait(s_full + g, ns, kSiteTreeSoftS)) break;
        ++ns;
        ptx::tc_fence_after();
        if (active) {
          if (masked) {  // -inf for what a row does not see (rolled: this code is cold)
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
              const int at = tok + 32 * u - C;  // draft number of the first of these columns
              const uint32_t sees = at >= 64    ? 0u
                                    : at >= 0   ? static_cast<uint32_t>(bits >> at)
                                    : at <= -32 ? 0xffffffffu
                                                : (static_cast<uint32_t>(bits << -at) | ((1u << -at) - 1u));
              uint32_t sv[32];
              ptx::tmem_ld32(s_tmem + 32 * u, sv);
              ptx::tmem_ld_wait();
              ptx::reg_fence32(sv);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(sees >> e & 1)) sv[e] = 0xff800000u;
              ptx::tmem_st32(s_tmem + 32 * u, sv);
            }
            ptx::tmem_st_wait();
          }
          // The row's maximum, three quarters of the scores on their way together (all four gain nothing, two 1-2%
          // slower with 256 rows); then P, a half at a time, of which the upper is still in registers (both halves
          // kept spill). Rolled: the code of four unrolled quarters pushes that of the MMA warp out of the
          // instruction cache.
          uint32_t sa[32], sb[32];
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = -INFINITY;
          auto fold = [&](const uint32_t(&v)[32]) {
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx8[(e >> 1) & 7] = ptx::fmax3(mx8[(e >> 1) & 7], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          };
          {
            uint32_t lower[32];
            ptx::tmem_ld32(s_tmem, lower);
            ptx::tmem_ld32(s_tmem + 64, sa);
            ptx::tmem_ld32(s_tmem + 96, sb);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(lower);
            ptx::reg_fence32(sa);
            ptx::reg_fence32(sb);
            fold(lower);
            ptx::tmem_ld32(s_tmem + 32, lower);
            fold(sa);
            fold(sb);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(lower);
            fold(lower);
          }
          const float mnew = fmaxf(ptx::fmax3(mx8[0], mx8[1], mx8[2]),
                                   ptx::fmax3(ptx::fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7])) * sl;
          if (t < step) {
            m = mnew;
          } else {
            // O is rescaled only when the running maximum grows by more than 2^8; otherwise the
            // old one stays the reference and P stays below 2^8.
            const bool need = row_ok && mnew > m + 8.0f;
            if (__any_sync(0xffffffffu, need)) {  // S of this tile is complete, so P V of the last one is
              const float mm = need ? mnew : m;
              const float f = need ? ptx::ex2(m - mm) : 1.f;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                ptx::tmem_ld32(o_tmem + g * D + 32 * c, ov);
                ptx::tmem_ld_wait();
                ptx::reg_fence32(ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                ptx::tmem_st32(o_tmem + g * D + 32 * c, ov);
              }
              l *= f;
              m = mm;
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;  // a row with no visible key yet keeps P = 0
          const uint64_t nmu2 = ptx::f2_packf(-mu, -mu);
          uint64_t ls2[4] = {0, 0, 0, 0};
          // P of 32 keys, over columns of S whose scores have been read: the upper half of S, in the keys' order
          auto exps = [&](const uint32_t(&v)[32], int u) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(v[2 * e], v[2 * e + 1]), sl2, nmu2), x0, x1);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              ls2[e & 3] = ptx::f2_add(ls2[e & 3], ptx::f2_packf(p0, p1));
              pk[e] = ptx::pack_bf16(p0, p1);  // off by up to 2^-8 of a weight; the sum takes it unrounded
            }
            ptx::tmem_st16(s_tmem + 64 + 16 * u, pk);
          };
#pragma unroll 1
          for (int half = 1; half >= 0; --half) {
            if (!half) {  // the upper ones are still here
              ptx::tmem_ld32(s_tmem, sa);
              ptx::tmem_ld32(s_tmem + 32, sb);
              ptx::tmem_ld_wait();
              ptx::reg_fence32(sa);
              ptx::reg_fence32(sb);
            }
            exps(sa, 2 * half);
            exps(sb, 2 * half + 1);
            if (half) {
              ptx::tmem_st_wait();
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(p_half + g);
            }
          }
          float a0, a1;
          ptx::f2_unpack(ptx::f2_add(ptx::f2_add(ls2[0], ls2[1]), ptx::f2_add(ls2[2], ls2[3])), a0, a1);
          l += a0 + a1;
        } else if (lane == 0) {
          ptx::mbar_arrive(p_half + g);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full + g);
      }
      if (!ok) break;
      // -------------------------------------------------------- the item's end
      const bool whole = I.t0 == 0 && I.t1 == I.nt;
      const int64_t slot = 2 * cta + (I.t0 > 0 ? 0 : 1);  // a CTA's first item may continue a line, its last one be cut
      const int mt = I.two ? g : 0;
      const int64_t out_row = row_ok ? static_cast<int64_t>(I.q0 + node) * p.hq + I.h * p.group + row_head : 0;
      float f0 = 0.f, f1 = 0.f, lse2 = -INFINITY;
      const bool both = !I.two && nt > 1;  // one row tile, two streams to join
      if ((I.two || g == 0 || both) && !wait(o_full + g, g ? no1 : no0, kSiteTreeSoftO)) break;
      if (I.two) {
        f0 = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN stays one
        lse2 = l == 0.f ? -INFINITY : m + log2f(l);
      } else {
        if (both || g == 0) {
          ml[g * kTile + r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ml_full + g);
        }
        float2 o0 = make_float2(m, l), o1 = make_float2(-INFINITY, 0.f);
        if (both || g == 1) {
          const int og = 1 - g;
          if (!wait(o_full + og, og ? no1 : no0, kSiteTreeSoftO)) break;
          if (!wait(ml_full + og, og ? nml1 : nml0, kSiteTreeSoftMl)) break;
          const float2 other = ml[og * kTile + r];
          if (g == 0) {
            o1 = other;
          } else {
            o1 = both ? o0 : o1;
            o0 = other;
          }
        }
        ++nml0;
        if (both) ++nml1;
        const float M = fmaxf(o0.x, o1.x), Mu = M == -INFINITY ? 0.f : M;
        const float w0 = ptx::ex2(o0.x - Mu), w1 = ptx::ex2(o1.x - Mu);
        const float sum = o0.y * w0 + o1.y * w1;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        f0 = w0 * inv;
        f1 = w1 * inv;
        lse2 = sum == 0.f ? -INFINITY : M + log2f(sum);
      }
      ++no0;
      if (I.two || both) ++no1;
      ptx::tc_fence_after();
      const uint64_t flagged = static_cast<uint64_t>(I.t1) * kTile > C ? (s_flags[it & 3] & bits) : 0;
      // two row tiles: a stream reads its own accumulator; else both halves of the columns are shared out
      const int c_begin = I.two ? 0 : g * kHalf, c_end = I.two ? D : c_begin + kHalf;
      if (active) {
        __nv_bfloat16* out_o = p.o + out_row * D;
        // [slot][row tile][D / 4][128 rows] of four columns: neighbouring lanes side by side
        float* out_part = p.w.part_o + ((slot * p.w.row_tiles + mt) * (D / 4) * kTile + r) * 4;
        int rows4[4];  // the rows of this lane's four lanes
#pragma unroll
        for (int k = 0; k < 4; ++k)
          rows4[k] = __shfl_sync(0xffffffffu, row_ok ? static_cast<int>(out_row) : -1, (lane & ~3) + k);
        // A weight of 0 multiplies too: a NaN or an infinity of V stays not finite however small its weight. (A row
        // that saw nothing has P = 0 and V without such values behind it, so its accumulator is 0.)
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 32) {
          uint32_t ov[32];
          ptx::tmem_ld32(o_tmem + (I.two ? g * D : 0) + c, ov);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(ov);
          float of[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) of[e] = __uint_as_float(ov[e]) * f0;
          if (both) {
            ptx::tmem_ld32(o_tmem + D + c, ov);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) of[e] += __uint_as_float(ov[e]) * f1;
          }
          if (!whole) {
            if (row_ok) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(out_part + (c + e) * kTile) = make_float4(of[e], of[e + 1], of[e + 2], of[e + 3]);
            }
          } else {
            // Four lanes exchange the 16-byte pieces of their four rows, so that a store writes 64 bytes of eight
            // rows and not 16 of 32 (a line a lane: 4600 cycles for two tiles of 128 rows, more than an own tile costs).
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = ptx::pack_bf16(of[2 * e], of[2 * e + 1]);
            const bool hi2 = lane & 2, hi1 = lane & 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // pieces 2, 3 of the lower pair against 0, 1 of the upper
              const uint32_t got = __shfl_xor_sync(0xffffffffu, hi2 ? w[e] : w[8 + e], 2);
              w[e] = hi2 ? got : w[e];
              w[8 + e] = hi2 ? w[8 + e] : got;
            }
#pragma unroll
            for (int q = 0; q < 16; q += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) {  // pieces 1 (3) of the even lane against 0 (2) of the odd
                const uint32_t got = __shfl_xor_sync(0xffffffffu, hi1 ? w[q + e] : w[q + 4 + e], 1);
                w[q + e] = hi1 ? got : w[q + e];
                w[q + 4 + e] = hi1 ? w[q + 4 + e] : got;
              }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (rows4[k] >= 0)
                ptx::st_v4(p.o + static_cast<int64_t>(rows4[k]) * D + c + 8 * (lane & 3), w[4 * k], w[4 * k + 1],
                           w[4 * k + 2], w[4 * k + 3]);
          }
        }
        __syncwarp();
        if (flagged) add_not_finite(p, I.b, I.h, C, flagged, D, c_begin, c_end, whole ? out_o : nullptr, out_part);
        if (row_ok && (I.two || g == 0)) {
          if (whole)
            p.lse[out_row] = lse2 * kLn2f;
          else
            p.w.part_lse2[(slot * p.w.row_tiles + mt) * kTile + r] = lse2;
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(o_free);
      ++it;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

// Joins the parts of the lines that were cut: lse = log2 sum 2^lse_p, O = sum 2^(lse_p - lse) O_p.
// Every block looks at all borders between the CTAs' ranges and lists those that are the first in their
// line; the listed lines, in pieces of 256 threads with four columns of a row each, are dealt out to the
// blocks. (A block for each border and piece, most of which had nothing to do, and two passes over the
// parts: 20 us against 8 for 8 lines of 19 parts and 240 rows.) The first block also gathers the CTAs' findings.
constexpr int kJoinThreads = 256, kJoinCtas = 512, kJoinAhead = 4, kJoinBlocks = 4;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_tree_join_kernel(const TreeParams p, int ctas_launched) {
  __shared__ int4 s_line[kJoinCtas], s_rest[kJoinCtas];  // (border, KV head, row group, parts), (-, first row, nodes, two)
  __shared__ int s_found[kJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_prior_grid();
  const uint32_t total = *p.w.total, ctas = min(static_cast<uint32_t>(ctas_launched), total);
  int lines = 0;
  for (uint32_t c0 = 1; c0 < ctas; c0 += kJoinThreads) {
    const uint32_t c = c0 + tid;
    int4 first = make_int4(0, 0, 0, 0), rest = first;
    if (c < ctas) {
      first = p.w.records[2 * c];
      rest = p.w.records[2 * c + 1];
    }
    const uint32_t line = c < ctas ? share_begin(total, ctas, c) - first.w : 0, end = line + rest.x;
    // a line goes on over the border, and no earlier border lies inside it
    const bool found = first.w > 0 && share_begin(total, ctas, c - 1) <= line;
    const uint32_t m = __ballot_sync(0xffffffffu, found);
    if (lane == 0) s_found[warp] = __popc(m);
    __syncthreads();
    int at = lines + __popc(m & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      at += w < warp ? s_found[w] : 0;
      lines += s_found[w];
    }
    if (found) {
      // how many shares begin before the line's end
      const uint32_t each = total / ctas, longer = total - each * ctas;
      const uint32_t before = end <= longer * (each + 1) ? (end + each) / (each + 1)
                                                         : longer + (end - longer * (each + 1) + each - 1) / each;
      s_line[at] = make_int4(c, first.y, first.z, static_cast<int>(min(before, ctas) - c) + 1);
      s_rest[at] = rest;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid < 32) {
    int code = 0, site = 0;
    for (int c = tid; c < ctas_launched; c += 32)
      if (code == 0 && p.w.cta_status[2 * c] != 0) {
        code = p.w.cta_status[2 * c];
        site = p.w.cta_status[2 * c + 1];
      }
    const uint32_t any = __ballot_sync(0xffffffffu, code != 0);
    const int src = any ? __ffs(any) - 1 : 0;
    code = __shfl_sync(0xffffffffu, code, src);
    site = __shfl_sync(0xffffffffu, site, src);
    for (int i = tid; i < static_cast<int>(kStatusBytes / 4); i += 32)
      p.w.status[i] = i == 0 ? code : (i == 1 ? site : 0);
  }
  const int pieces = p.w.row_tiles * (D / 4) * kTile / kJoinThreads;  // of a line: [row tile][D / 4][128 rows]
  for (int w = blockIdx.x; w < lines * pieces; w += gridDim.x) {
    const int4 line = s_line[w / pieces], rest = s_rest[w / pieces];
    const int item = w % pieces * kJoinThreads + tid;
    const int r = item & (kTile - 1), chunk = (item >> 7) % (D / 4), mt = (item >> 7) / (D / 4);
    const int row_node = r / p.group, node = (2 * line.z + mt) * p.nodes_per_tile + row_node;
    if (mt > rest.w || row_node >= p.nodes_per_tile || node >= rest.z) continue;
    // the parts: the last item of CTA c - 1, then the first ones of c, c + 1, .. up to the line's end
    const int c = line.x, parts = line.w;
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += kJoinAhead) {
      float lse[kJoinAhead];
      float4 o[kJoinAhead];
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const int i = i0 + e;
        lse[e] = -INFINITY;
        if (i < parts) {
          const int64_t slot = (i == 0 ? 2 * c - 1 : 2 * (c - 1 + i)) * static_cast<int64_t>(p.w.row_tiles) + mt;
          lse[e] = p.w.part_lse2[slot * kTile + r];
          o[e] = reinterpret_cast<const float4*>(p.w.part_o)[(slot * (D / 4) + chunk) * kTile + r];
        }
      }
      float top = M;
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) top = fmaxf(top, lse[e]);
      const float ref = top == -INFINITY ? 0.f : top, f = ptx::ex2(M - ref);  // M = -inf: 0
      sum *= f;
      acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const float wt = ptx::ex2(lse[e] - ref);  // no such part: 0
        sum += wt;
        // a part whose weight is 0 counts: 0 * NaN, and 0 * infinity, are NaN
        if (i0 + e < parts) acc.x += wt * o[e].x, acc.y += wt * o[e].y, acc.z += wt * o[e].z, acc.w += wt * o[e].w;
      }
      M = top;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = static_cast<int64_t>(rest.y + node) * p.hq + line.y * p.group + r % p.group;
    *reinterpret_cast<uint2*>(p.o + row * D + 4 * chunk) =
        make_uint2(ptx::pack_bf16(acc.x * inv, acc.y * inv), ptx::pack_bf16(acc.z * inv, acc.w * inv));
    if (chunk == 0) p.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2f;
  }
}

template <int D>
cudaError_t launch_tree_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                          int grid, void* events, cudaStream_t stream) {
  if (grid > kJoinCtas) grid = kJoinCtas;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(decode_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TreeLayout<D>::kBytes);
  });
  if (e != cudaSuccess) return e;
  cudaEvent_t* ev = static_cast<cudaEvent_t*>(events);
  if (ev) cudaEventRecord(ev[0], stream);
  decode_tree_kernel<D><<<grid, kTreeThreads, TreeLayout<D>::kBytes, stream>>>(tq, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (ev) cudaEventRecord(ev[1], stream);
  return launch_after(decode_tree_join_kernel<D>, dim3(kJoinBlocks * grid), dim3(kJoinThreads), 0, stream, p, grid);
}

}  // namespace

cudaError_t launch_decode_tree(const jfa_decode_tree_args& a, const TreeBuffers& w, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv, int box, uint64_t budget_ns, int grid,
                               cudaStream_t stream) {
  TreeParams p{};
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.q_offsets = a.q_offsets;
  p.mask = a.tree_mask;
  p.k_cache = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.w = w;
  p.batch = a.batch;
  p.hq = a.q_heads;
  p.hkv = a.kv_heads;
  p.group = a.q_heads / a.kv_heads;
  p.page = make_fast_div(a.page_size);
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.total_q = a.total_q;
  p.max_q = a.max_q;
  p.nodes_per_tile = tree_nodes_per_tile(p.group);
  p.node_tile_mul = 65536u / static_cast<uint32_t>(p.nodes_per_tile) + 1;
  p.box = box;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.budget_ns = budget_ns;
  return a.head_dim == 128 ? launch_tree_d<128>(tq, tk, tv, p, grid, a.main_kernel_events, stream)
                           : launch_tree_d<64>(tq, tk, tv, p, grid, a.main_kernel_events, stream);
}

}  // namespace jfa
