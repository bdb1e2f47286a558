// Decode over the 8-bit paged KV cache: the last q_len tokens of each sequence
// attend to its e4m3 keys and values, each block of tokens and head with its
// own scale; optionally every cached token's attention weight is added to a
// running sum (what eviction goes by).
//
// Mathematics, for one sequence and KV head, rows r = (query token, head of the
// group), tokens t, in units of log2 (c = scale * log2 e):
//   s_rt = c * ks_t * sum_d q_rd k_td       (k, v: e4m3 values; ks, vs: scales)
//   p_rt = 2^(s_rt - m_r), l_r = sum_t p_rt, m_r a running reference
//   w_rt = 2^(s_rt + log2 vs_t - n_r), O_r = 2^(n_r - m_r) / l_r * sum_t w_rt v_t
// V's scale goes into the exponent of a second weight w with a reference n of
// its own, so that w spans the full fp16 range whatever the scales are.
//
// Design (GB300). The path is bound by HBM: 2 (D + 4 / block) bytes per token
// and head for 4 D flops per row, about 4 flop per byte at 8 rows. What the
// kernel has to spare is issue slots, since a code byte is half the traffic
// of a bf16 one and needs a conversion more:
//  * Tokens are the M side of the register MMAs (m16n8k16, fp16, fp32
//    accumulators): S^T = K Q^T and O^T = V^T P^T. A group of up to 8 rows
//    fills N exactly, half the MMAs of rows on the M side; 9..16 rows take two
//    N halves that share the converted operands. tcgen05 would pad 8 rows to
//    its M of 64 or 128 and needs the operand in shared memory as 16-bit data,
//    which would cost a write and a read of twice the code bytes.
//  * Codes convert to fp16 exactly. Q goes to fp16 after a division by a power
//    of two per row (its largest value becomes 1..2); P is rounded to fp16,
//    2^-11 relative, an eighth of the bf16 output's own rounding.
//  * The references m and n are raised only when a score passes them by 2^8
//    (a warp vote); the usual tile has no reduction over lanes and no rescale.
//    w stays below 2^15 and its reference starts 2^7 below the largest weight,
//    so fp16 keeps weights down to 2^-31 of it.
//  * Copies are cp.async, 16 bytes a lane, eight neighbouring lanes on one
//    128-byte line: the rate of reads follows the number of lines that a
//    quarter of a warp touches (measured on 1.08 GB of rows behind a page
//    table: one line 6.7-7.0 TB/s, four half or quarter lines 5.2 TB/s).
//  * Warps are independent. Work is split evenly whatever the lengths: the
//    16-token tiles of all sequences form one line, cut into equal parts; a
//    group of kv_heads consecutive warps takes a part, one head each, so the
//    heads of a token, neighbours in memory, are read at about the same time.
//    A warp that meets a sequence's end writes what it has and goes on, with
//    the next sequence's tiles already on their way. A sequence inside one part
//    is finished there; one that was cut leaves a partial result per part,
//    joined by a second kernel in the order of the parts (no atomics on
//    results: the outcome depends on the lengths and the SM count only).
//
// Index mappings (each lane: g = lane / 4, q = lane % 4):
//  * K: the A operand's rows are tokens g and g + 8; the head dimension is
//    permuted so that a lane's four k-values of step (c, w) are the bytes
//    64 c + 16 q + 4 w .. + 3; Q is loaded with the same permutation.
//  * V: the A operand's rows are head dimensions; row g of step j is dimension
//    (D/8) g + 2 j and row g + 8 the next one, so a lane reads D/8 contiguous
//    bytes of tokens 2q, 2q + 1, 2q + 8, 2q + 9. The accumulator then holds
//    those D/8 dimensions of query rows 2q and 2q + 1.
//  * P: S^T's accumulator (rows = tokens) becomes the B operand (columns =
//    query rows) by an 8 x 8 transposition between lanes (movmatrix).
//  * Shared memory: 128-byte lines of 16-byte pieces; piece i of line n lies at
//    i ^ f(n), with f chosen so that eight lanes of a read, which touch two
//    lines (K) or four (V), meet no bank twice.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fp8_cache.cuh"

namespace jfa {

struct Fp8DecodeParams {
  const __nv_bfloat16* q;
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  int32_t batch, hq, group, q_len, max_pages, page_size;
  float scale_log2;
  int32_t* tile_base;  // [B + 1] 16-token tiles of the sequences before b
  int32_t* long_list;  // how many sequences are cut into too many parts for a warp to join a row, and which
  int32_t max_parts;   // most parts of the line
  int32_t grid;        // blocks of the main kernel (four warps each)
  FastDiv by_heads;    // division by hkv
  uint8_t* errors;     // a byte for each warp of the main kernel (pages), then a 32-bit word (lengths)
  float* part_o;       // [parts + B][hkv][rows][D], normalised
  float* part_lse2;    // [parts + B][hkv][rows], log2, -inf when empty
  __nv_bfloat16* o;
  float* lse;          // [B, q_len, Hq] natural log
  float* lse2;         // [B, hkv, rows] log2, +inf where a row sees no key (weights only)
  float* scores;       // [tiles][hkv][rows][16] log2 units (weights only)
  const float* w_in;   // [B, hkv, max_pages * page_size] or null
  float* w_out;
  float decay;
  int32_t* status;
};

constexpr int kF8Warps = 4;
// Batches up to this number their tiles in every block, larger ones in a kernel before: 512 x 100-1000
// tokens of one KV head of 64 18.1 against 19.8 us, 256 x 13.9 against 16.1; 1024 x 27.4 against 27.6,
// for 4 KB more of shared memory.
constexpr int kF8ScanBatch = 512;
constexpr int kF8RowParts = 62;   // parts that a warp joins a row of (two lse a lane, less two shared parts)
// A score may pass its reference by this much before the reference moves.
constexpr float kF8Slack = 8.f;
// w's reference lies this far below the largest s + log2 vs when it is set.
constexpr float kF8WShift = 7.f;
constexpr float kF8NoRef = -3.0e38f;  // a reference before the first visible token

template <int D, int NR>
struct F8Tile {
  // By the registers: 128 a thread, or 255 with 16 rows; at head_dim 128 one to three of them
  // spill (4 to 12 bytes). (16 rows at head_dim 128 in 168 registers spill far more, 88 us against
  // 67 us for 16 x 0.5k-8k tokens with 4 query tokens of 4 heads; with Q in shared memory instead
  // of 32 of the registers they take 70 us.)
  static constexpr int kCtasPerSm = NR == 1 ? 4 : 2;
  // Tiles computed together. 16 rows leave 8 warps an SM, too few to cover the chain of a tile's
  // steps by each other's work: two tiles give each warp two such chains.
  static constexpr int kTogether = NR;
  // One tile on its way while one is computed, per warp: with 16 warps that is
  // 68 KB an SM. More queue up in front of the memory: 32 x 1k-32k tokens, NR 1,
  // take 175 us with 2 stages and 187 us with 3. With 8 warps that is two, and two computed.
  static constexpr int kStages = NR == 1 ? 2 : 4;
  static constexpr int kVOff = 16 * D;           // K rows, V rows, 16 + 16 scales
  static constexpr int kScaleOff = 32 * D;
  static constexpr int kStageBytes = kScaleOff + 128;
  static constexpr int kRingBytes = kF8Warps * kStages * kStageBytes;
};

// Codes are read once: they make way first in L2, for the parts' results and the
// scores that the next kernels read (one sequence of 131k tokens 51 -> 48 us, four
// draft tokens with weights 60 -> 54 us).
__device__ __forceinline__ uint64_t f8_read_once() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void f8_cp_async16(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void f8_cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void f8_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void f8_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void f8_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f8_pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// log2 of a scale (0, for a missing token, gives -inf).
__device__ __forceinline__ float f8_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 x 8 matrix of 16-bit elements, transposed between the lanes of a warp.
__device__ __forceinline__ uint32_t f8_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A row that sees no key counts nothing for the weights: its lse is kept as +inf there.
__device__ __forceinline__ float f8_weight_lse(float z) { return z == -INFINITY ? INFINITY : z; }

// A sequence's length, 0 where it is out of range.
__device__ __forceinline__ int f8_length(const Fp8DecodeParams& p, int b, bool* bad) {
  const int L = p.seqlens[b];
  *bad = L < 0 || L > static_cast<int64_t>(p.max_pages) * p.page_size || (L > 0 && p.c.num_pages == 0);
  return *bad ? 0 : L;
}

// Numbers the tiles: base[b] = sum over b' < b of ceil(L_b' / 16), b = 0 .. batch;
// len, if given, receives the lengths. Every thread of the block takes part; true
// if a length was out of range.
template <int THREADS>
__device__ __forceinline__ bool f8_number_tiles(const Fp8DecodeParams& p, int32_t* base, int32_t* len = nullptr) {
  __shared__ int32_t warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) base[0] = 0;
  int running = 0;
  bool any = false;
  for (int b0 = 0; b0 < p.batch; b0 += THREADS) {
    int x = 0;
    if (b0 + tid < p.batch) {
      bool bad;
      const int L = f8_length(p, b0 + tid, &bad);
      if (len) len[b0 + tid] = L;
      x = (L + 15) >> 4;
      any |= bad;
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = running;
    for (int w = 0; w < THREADS / 32; ++w) {
      const int y = warp_sum[w];
      before += w < warp ? y : 0;
      running += y;
    }
    if (b0 + tid < p.batch) base[b0 + tid + 1] = before + x;
    __syncthreads();
  }
  return __syncthreads_or(any);
}

// The line of tiles, cut into parts of equal length.
struct F8Line {
  int64_t total;  // tiles of all sequences
  int64_t parts;  // parts in use
  __device__ __forceinline__ F8Line(int32_t tiles, int max_parts) {
    total = tiles;
    parts = min(static_cast<int64_t>(max_parts), total);
  }
  __device__ __forceinline__ int begin(int64_t i) const { return quotient(static_cast<uint64_t>(i * total), parts); }
  // the part that holds tile x: the last i with floor(i total / parts) <= x
  __device__ __forceinline__ int part_of(int64_t x) const {
    return quotient(static_cast<uint64_t>((x + 1) * parts - 1), total);
  }
  // A long sequence: of more than 62 parts (64 with what its ends share with others').
  __device__ __forceinline__ bool is_long(int base, int end) const { return (end - base) * parts > kF8RowParts * total; }
  // n / d, in 32 bits where both fit (a 64-bit division is a hundred instructions)
  static __device__ __forceinline__ int quotient(uint64_t n, int64_t d) {
    return static_cast<int>(n >> 32 ? n / static_cast<uint64_t>(d) : static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
  }
};

// Lists the long sequences (fewer than 64: the parts are at most kFp8MaxWarps).
static_assert(kFp8MaxWarps / kF8RowParts < kFp8LongList - 1, "the list holds them all");
template <int THREADS>
__device__ __forceinline__ void f8_list_long(const Fp8DecodeParams& p, const int32_t* base) {
  __shared__ int32_t s_count;
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  const F8Line line(base[p.batch], p.max_parts);
  for (int b = threadIdx.x; b < p.batch; b += THREADS)
    if (line.is_long(base[b], base[b + 1])) p.long_list[1 + atomicAdd(&s_count, 1)] = b;
  __syncthreads();
  if (threadIdx.x == 0) p.long_list[0] = s_count;
}

// Large batches: one block numbers the tiles for all.
__global__ void __launch_bounds__(1024) fp8_decode_plan_kernel(const Fp8DecodeParams p) {
  allow_next_grid();
  const bool bad = f8_number_tiles<1024>(p, p.tile_base);
  f8_list_long<1024>(p, p.tile_base);
  if (threadIdx.x == 0) reinterpret_cast<uint32_t*>(p.errors)[p.grid] = bad;
}

// The sequence that holds tile x, from sequence `from` on: the warp's lanes look at 32 bounds at a
// time, first far apart, so that a batch padded with empty sequences costs little more than
// without them (of 2048 sequences 8 with 0.5k-7k tokens: 53 us, 83 us one bound after the other).
__device__ __forceinline__ int f8_find_sequence(const int32_t* tile_base, int batch, int x, int from) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = from, n = batch - from;
  while (n > 32) {
    const uint32_t step = (n + 31) >> 5, end = min(lo + (lane + 1) * step, static_cast<uint32_t>(batch));
    const uint32_t m = __ballot_sync(0xffffffffu, tile_base[end] > x);
    lo += (m ? __ffs(m) - 1 : 31) * step;
    n = min(step, batch - lo);
  }
  const uint32_t m = __ballot_sync(0xffffffffu, lane < n && tile_base[lo + lane + 1] > x);
  return m ? static_cast<int>(lo) + __ffs(m) - 1 : batch - 1;
}
// The next sequence after b that holds tile x, most often b + 1.
__device__ __forceinline__ int f8_next_sequence(const int32_t* tile_base, int batch, int x, int b) {
  ++b;
  return tile_base[b + 1] > x ? b : f8_find_sequence(tile_base, batch, x, b);
}

template <int D, int NR, bool WEIGHTS>
__global__ void __launch_bounds__(128, F8Tile<D, NR>::kCtasPerSm) fp8_decode_kernel(const Fp8DecodeParams p) {
  using T = F8Tile<D, NR>;
  constexpr int kSteps = D / 16;  // MMA steps of Q K^T, and of P V
  constexpr int kEpl = D / 8;     // head dimensions a lane holds of each of its query rows
  constexpr int kStages = T::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t s_base[kF8ScanBatch + 1], s_len[kF8ScanBatch];

  const int32_t* tile_base = p.tile_base;
  if (p.batch <= kF8ScanBatch) {
    const bool bad = f8_number_tiles<128>(p, s_base, s_len);
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i <= p.batch; i += 128) p.tile_base[i] = s_base[i];
      if (threadIdx.x == 0) reinterpret_cast<uint32_t*>(p.errors)[p.grid] = bad;
      f8_list_long<128>(p, s_base);
    }
    tile_base = s_base;
  } else {
    wait_prior_grid();  // the plan
  }
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, qq = lane & 3;
  const int hkv = p.c.hkv, G = p.group, QL = p.q_len, nrows = G * QL;
  const F8Line line(tile_base[p.batch], p.max_parts);
  const int jobs = static_cast<int>(line.parts) * hkv;  // at most the larger of the warps and hkv
  auto length = [&](int b) -> int {
    bool bad;
    return p.batch <= kF8ScanBatch ? s_len[b] : f8_length(p, b, &bad);
  };
  uint8_t* ring = smem + warp * kStages * T::kStageBytes;
  const uint32_t ring_u32 = ptx::smem_u32(ring);
  const uint64_t read_once = f8_read_once();
  bool bad_page = false;

  // Where this lane's copies of step u go: token tk(u), 16-byte piece cp of its row.
  constexpr int kLanesPerRow = D / 16, kCopies = D / 32;
  const int cp = lane % kLanesPerRow;
  auto copy_token = [&](int u) { return u * (32 / kLanesPerRow) + lane / kLanesPerRow; };
  auto k_place = [&](int tk) -> uint32_t {  // byte offset of piece cp of token tk's key
    if constexpr (D == 128) return tk * 128 + ((cp ^ ((tk & 1) << 2)) << 4);
    return tk * 64 + (cp << 4);
  };
  auto v_place = [&](int tk) -> uint32_t {
    if constexpr (D == 128) return tk * 128 + ((cp ^ (tk & 6)) << 4);
    return (tk >> 1) * 128 + (((((tk & 1) << 2) | cp) ^ (tk & 6)) << 4);
  };

  for (int job = blockIdx.x * kF8Warps + warp; job < jobs; job += gridDim.x * kF8Warps) {
    const int part = fast_div(job, p.by_heads), h = job - part * hkv;
    const int x0 = line.begin(part), x1 = line.begin(part + 1);
    int b = f8_find_sequence(tile_base, p.batch, x0, 0);

    // ---- producer: pages are looked up one tile before they are copied from
    int pb = b, pL = 0, pbase = 0, pend = 0;  // its sequence, length, first tile, end
    const int32_t* ppt = nullptr;
    int page = 0, slot = -1;  // of this lane's token (lane % 16) of the tile to copy next
    auto enter = [&]() {
      pL = length(pb);
      pbase = tile_base[pb];
      pend = tile_base[pb + 1];
      ppt = p.page_table + static_cast<int64_t>(pb) * p.max_pages;
    };
    auto look_up = [&](int x) {
      slot = -1;
      if (x < x1) {
        if (x >= pend) {
          pb = f8_next_sequence(tile_base, p.batch, x, pb);
          enter();
        }
        const int tok = (x - pbase) * 16 + (lane & 15);
        if (tok < pL) {
          const int pg = fast_div(tok, p.c.page);
          page = ppt[pg];
          slot = tok - pg * p.page_size;
        }
      }
    };
    auto issue = [&](int i) {
      if (x0 + i < x1) {
        int row = -1;  // cache row of the token, -1 past the end of the sequence
        if (slot >= 0) {
          if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.num_pages)) {
            bad_page = true;
            page = 0;
          }
          row = page * p.page_size + slot;
        }
        const uint32_t st = ring_u32 + (i % kStages) * T::kStageBytes;
        const int64_t sc = static_cast<int64_t>(max(row, 0) >> p.c.block_shift) * hkv + h;
        f8_cp_async4(st + T::kScaleOff + lane * 4, (lane < 16 ? p.c.ks : p.c.vs) + sc, row >= 0 ? 4 : 0);
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          const int tk = copy_token(u);
          const int r = __shfl_sync(0xffffffffu, row, tk);
          const int64_t off = (static_cast<int64_t>(max(r, 0)) * hkv + h) * D + cp * 16;
          const uint32_t n = r >= 0 ? 16 : 0;  // missing tokens are zeros
          f8_cp_async16(st + k_place(tk), p.c.kc + off, n, read_once);
          f8_cp_async16(st + T::kVOff + v_place(tk), p.c.vc + off, n, read_once);
        }
      }
      f8_commit();  // one group per call, empty past the last tile
    };
    enter();
    look_up(x0);
    for (int i = 0; i < kStages - T::kTogether; ++i) {
      issue(i);
      look_up(x0 + i + 1);
    }

    for (int x = x0; x < x1;) {
      // ---- the sequence b, from tile t_lo on
      if (tile_base[b + 1] <= x) b = f8_next_sequence(tile_base, p.batch, x, b);
      const int L = length(b);
      const int base = tile_base[b], end = tile_base[b + 1];
      const int x_first = x, x_stop = min(end, x1);

      // ---- Q as the B operand: column g of half u is row 8 u + g, scaled to 1..2
      uint32_t qb[NR][kSteps][2];
      float rq[NR][2];  // factors of the scores of rows 2q and 2q + 1 of each half
      int lim[NR][2];   // their causal limits: tokens below are visible
#pragma unroll
      for (int u = 0; u < NR; ++u) {
        const int r = 8 * u + gq;
        const bool real = r < nrows;
        const __nv_bfloat16* qr = p.q + ((static_cast<int64_t>(b) * QL + (real ? r / G : 0)) * p.hq +
                                         static_cast<int64_t>(h) * G + (real ? r % G : 0)) * D;
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real) v = *reinterpret_cast<const uint4*>(qr + 64 * c + 16 * qq + 8 * e);
            const uint32_t raw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // element 8 e + 2 k of the 16 is step w = 2 e + k / 2, register k % 2
              qb[u][4 * c + 2 * e + (k >> 1)][k & 1] = raw[k];
              const float a0 = fabsf(ptx::bf16lo(raw[k])), a1 = fabsf(ptx::bf16hi(raw[k]));
              if (a0 < INFINITY) amax = fmaxf(amax, a0);
              if (a1 < INFINITY) amax = fmaxf(amax, a1);
            }
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^-e and 2^e of the row's exponent, kept within the normal range
        const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qb[u][s][e] = f8_pack_f16(ptx::bf16lo(qb[u][s][e]) * down, ptx::bf16hi(qb[u][s][e]) * down);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          rq[u][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * qq + e)) * p.scale_log2;
          lim[u][e] = L - QL + (8 * u + 2 * qq + e) / G + 1;
        }
      }
      const int lim_min = L - QL + 1;  // the earliest query token's limit

      float m[NR][2], n[NR][2], l[NR][2], acc[NR][kSteps][4];
#pragma unroll
      for (int u = 0; u < NR; ++u) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[u][e] = n[u][e] = kF8NoRef;
          l[u][e] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) acc[u][j][0] = acc[u][j][1] = acc[u][j][2] = acc[u][j][3] = 0.f;
      }

      // ---- N neighbouring tiles, from tile x of the line on
      auto step = [&](auto tag) {
        constexpr int N = decltype(tag)::value;
        const int i = x - x0;
        __syncwarp();  // every lane has read the slots that are refilled now
#pragma unroll
        for (int t = 0; t < N; ++t) {
          issue(i + kStages - T::kTogether + t);
          look_up(x + kStages - T::kTogether + t + 1);
        }
        f8_wait<kStages - T::kTogether>();  // this lane's copies of the N tiles have landed
        __syncwarp();                       // and the other lanes'
        const uint8_t* st[N];
        int t0[N];
        float ks[N][2], lv[N][2], s[N][NR][4];
#pragma unroll
        for (int t = 0; t < N; ++t) {
          st[t] = ring + ((i + t) % kStages) * T::kStageBytes;
          t0[t] = (x + t - base) * 16;
          const float* sc = reinterpret_cast<const float*>(st[t] + T::kScaleOff);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[t][e] = sc[gq + 8 * e];
            lv[t][e] = f8_log2(sc[16 + gq + 8 * e]);
          }
        }

        // S^T = K Q^T
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
          for (int u = 0; u < NR; ++u) s[t][u][0] = s[t][u][1] = s[t][u][2] = s[t][u][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 k0[N], k1[N];
#pragma unroll
          for (int t = 0; t < N; ++t) {
            const uint8_t* src = D == 128 ? st[t] + gq * 128 + (((qq + 4 * c) ^ ((gq & 1) << 2)) << 4)
                                          : st[t] + gq * 64 + (qq << 4);
            k0[t] = *reinterpret_cast<const uint4*>(src);
            k1[t] = *reinterpret_cast<const uint4*>(src + 8 * D);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int t = 0; t < N; ++t) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(w == 0 ? k0[t].x : (w == 1 ? k0[t].y : (w == 2 ? k0[t].z : k0[t].w)), a0, a2);
              e4m3x4_to_f16(w == 0 ? k1[t].x : (w == 1 ? k1[t].y : (w == 2 ? k1[t].z : k1[t].w)), a1, a3);
#pragma unroll
              for (int u = 0; u < NR; ++u) f8_mma(s[t][u], a0, a1, a2, a3, qb[u][4 * c + w][0], qb[u][4 * c + w][1]);
            }
        }
        // scaled scores: s[..][0..1] token g, rows 2q and 2q + 1; s[..][2..3] token g + 8
        const bool partial = t0[N - 1] + 16 > lim_min;
        bool raise = false;
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
          for (int u = 0; u < NR; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[t][u][e] *= ks[t][0] * rq[u][e];
              s[t][u][2 + e] *= ks[t][1] * rq[u][e];
              if (partial) {
                if (t0[t] + gq >= lim[u][e]) s[t][u][e] = -INFINITY;
                if (t0[t] + gq + 8 >= lim[u][e]) s[t][u][2 + e] = -INFINITY;
              }
              raise |= fmaxf(s[t][u][e], s[t][u][2 + e]) > m[u][e] + kF8Slack;
              raise |= fmaxf(s[t][u][e] + lv[t][0], s[t][u][2 + e] + lv[t][1]) > n[u][e] + (kF8WShift + kF8Slack);
            }
        if constexpr (WEIGHTS) {
#pragma unroll
          for (int t = 0; t < N; ++t) {
            float* out = p.scores + (static_cast<int64_t>(x + t) * hkv + h) * nrows * 16;
#pragma unroll
            for (int u = 0; u < NR; ++u)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = 8 * u + 2 * qq + e;
                if (r < nrows) {
                  out[r * 16 + gq] = s[t][u][e];
                  out[r * 16 + gq + 8] = s[t][u][2 + e];
                }
              }
          }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int u = 0; u < NR; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float a = -INFINITY, c = -INFINITY;
#pragma unroll
              for (int t = 0; t < N; ++t) {
                a = fmaxf(a, fmaxf(s[t][u][e], s[t][u][2 + e]));
                c = fmaxf(c, fmaxf(s[t][u][e] + lv[t][0], s[t][u][2 + e] + lv[t][1]));
              }
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, off));
              }
              const float mn = fmaxf(m[u][e], a), nn = fmaxf(n[u][e], c - kF8WShift);
              l[u][e] *= ptx::ex2(m[u][e] - mn);
              const float f = ptx::ex2(n[u][e] - nn);
              m[u][e] = mn;
              n[u][e] = nn;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                acc[u][j][e] *= f;
                acc[u][j][2 + e] *= f;
              }
            }
        }
        // P^T as the B operand
        uint32_t pt2[N][NR][2];
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
          for (int u = 0; u < NR; ++u) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              l[u][e] += ptx::ex2(s[t][u][e] - m[u][e]) + ptx::ex2(s[t][u][2 + e] - m[u][e]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              pt2[t][u][k] = f8_transpose(f8_pack_f16(ptx::ex2(s[t][u][2 * k] + lv[t][k] - n[u][0]),
                                                      ptx::ex2(s[t][u][2 * k + 1] + lv[t][k] - n[u][1])));
          }
        // O^T += V^T P^T
        uint32_t vw[N][4][kEpl / 4];
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint8_t* vt = st[t] + T::kVOff;
            if constexpr (D == 128) {  // token 2q + (w & 1) + 8 (w / 2), piece g
              const uint4 v = *reinterpret_cast<const uint4*>(vt + (2 * qq + (w & 1) + 8 * (w >> 1)) * 128 +
                                                              ((gq ^ (2 * qq)) << 4));
              vw[t][w][0] = v.x;
              vw[t][w][1] = v.y;
              vw[t][w][2] = v.z;
              vw[t][w][3] = v.w;
            } else {  // line q + 4 (w / 2), half w & 1, piece g / 2, its half g & 1
              const uint2 v = *reinterpret_cast<const uint2*>(vt + (qq + 4 * (w >> 1)) * 128 +
                                                              (((((w & 1) << 2) | (gq >> 1)) ^ (2 * qq)) << 4) +
                                                              ((gq & 1) << 3));
              vw[t][w][0] = v.x;
              vw[t][w][1] = v.y;
            }
          }
        if (partial && QL > 1) {
          // A value that some rows may not see must not reach them even as
          // 0 * NaN: NaN codes leave V and are put into the rows that do see
          // them, where a second product counts them.
#pragma unroll
          for (int t = 0; t < N; ++t) {
            bool bad_v = false;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
              for (int k = 0; k < kEpl / 4; ++k) bad_v |= e4m3_any_nan(vw[t][w][k]);
            if (!__any_sync(0xffffffffu, bad_v)) continue;
            uint32_t one[4][kEpl / 4];  // e4m3 1.0 (0x38) where the code is NaN
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
              for (int k = 0; k < kEpl / 4; ++k) {
                const uint32_t hit = (((vw[t][w][k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 a byte
                one[w][k] = hit * 0x38u;
                vw[t][w][k] &= ~(hit * 0xFFu);
              }
#pragma unroll
            for (int u = 0; u < NR; ++u) {
              float see[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                see[e] = t0[t] + gq < lim[u][e] ? 1.f : 0.f;
                see[2 + e] = t0[t] + gq + 8 < lim[u][e] ? 1.f : 0.f;
              }
              const uint32_t b0 = f8_transpose(f8_pack_f16(see[0], see[1]));
              const uint32_t b1 = f8_transpose(f8_pack_f16(see[2], see[3]));
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(__byte_perm(one[0][j >> 1], one[1][j >> 1], sel), a0, a1);
                e4m3x4_to_f16(__byte_perm(one[2][j >> 1], one[3][j >> 1], sel), a2, a3);
                float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                f8_mma(cnt, a0, a1, a2, a3, b0, b1);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (cnt[e] > 0.f) acc[u][j][e] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            // bytes (token a, d), (token a + 1, d), (token a, d + 1), (token a + 1, d + 1)
            const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(__byte_perm(vw[t][0][j >> 1], vw[t][1][j >> 1], sel), a0, a1);
            e4m3x4_to_f16(__byte_perm(vw[t][2][j >> 1], vw[t][3][j >> 1], sel), a2, a3);
#pragma unroll
            for (int u = 0; u < NR; ++u) f8_mma(acc[u][j], a0, a1, a2, a3, pt2[t][u][0], pt2[t][u][1]);
          }
        x += N;
      };
      if constexpr (T::kTogether == 2)
        while (x + 1 < x_stop) step(std::integral_constant<int, 2>{});
      while (x < x_stop) step(std::integral_constant<int, 1>{});

      // ---- the end of the sequence, or of the part
      const bool whole = x_first == base && x_stop == end;
#pragma unroll
      for (int u = 0; u < NR; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[u][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const int r = 8 * u + 2 * qq + e;
          if (r >= nrows) continue;
          // a row that saw no token: zeros and -inf (NaN stays NaN)
          // 2^(n - m) / sum in two factors: with values of 2^-126 the whole would leave fp32's range
          const float half = ptx::ex2(0.5f * (n[u][e] - m[u][e])), f = sum == 0.f ? 0.f : half / sum;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            acc[u][j][e] *= half;
            acc[u][j][2 + e] *= half;
          }
          const float z = sum == 0.f ? -INFINITY : m[u][e] + log2f(sum);
          if (whole) {
            const int64_t row = (static_cast<int64_t>(b) * QL + r / G) * p.hq + static_cast<int64_t>(h) * G + r % G;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + kEpl * gq);
#pragma unroll
            for (int j = 0; j < kSteps; j += 4)
              *reinterpret_cast<uint4*>(dst + j) =
                  make_uint4(ptx::pack_bf16(acc[u][j][e] * f, acc[u][j][2 + e] * f),
                             ptx::pack_bf16(acc[u][j + 1][e] * f, acc[u][j + 1][2 + e] * f),
                             ptx::pack_bf16(acc[u][j + 2][e] * f, acc[u][j + 2][2 + e] * f),
                             ptx::pack_bf16(acc[u][j + 3][e] * f, acc[u][j + 3][2 + e] * f));
            if (gq == 0) {
              p.lse[row] = z * 0.6931471805599453f;
              if (WEIGHTS) p.lse2[(static_cast<int64_t>(b) * hkv + h) * nrows + r] = f8_weight_lse(z);
            }
          } else {
            const int64_t row = ((static_cast<int64_t>(part) + b) * hkv + h) * nrows + r;
            float* dst = p.part_o + row * D + kEpl * gq;
#pragma unroll
            for (int j = 0; j < kSteps; j += 2)
              *reinterpret_cast<float4*>(dst + 2 * j) =
                  make_float4(acc[u][j][e] * f, acc[u][j][2 + e] * f, acc[u][j + 1][e] * f, acc[u][j + 1][2 + e] * f);
            if (gq == 0) p.part_lse2[row] = z;
          }
        }
    }
    f8_wait<0>();
    __syncwarp();  // the ring is filled again for the next job
  }
  bad_page = __any_sync(0xffffffffu, bad_page);
  if (lane == 0) p.errors[blockIdx.x * kF8Warps + warp] = bad_page;
}

// Joins the parts of the sequences that were cut:
//   lse = log2 sum_i 2^lse_i, O = sum_i 2^(lse_i - lse) O_i,
// in a fixed order; a sequence without tokens gets zeros and -inf. The last block
// gathers the main kernel's findings into the status block.
// Two shapes. kWide = false: a warp per output row, for many sequences of a dozen
// parts or so: the lanes hold the parts' lse, and the first sixteen parts' rows are
// on their way before the lse are there (24 x 37-4k tokens of head_dim 64, 25 parts
// a sequence: 21.1 us the call, 21.9 with eight). The long sequences among them, which the
// main kernel has listed, are joined by all blocks together, as in the other shape
// (131k tokens and 79 x 500 of one KV head, 8 rows, with weights: 36 us, 171 us with one block a row).
// kWide = true: a block per 32 columns of a row, its 32 groups of eight lanes
// reading a part's 128-byte piece each, four ahead, so that a sequence cut into
// hundreds of parts is joined by all SMs.
template <int THREADS>
__device__ __forceinline__ void f8_report(const Fp8DecodeParams& p) {
  constexpr int kLoads = (kFp8MaxWarps / kF8Warps + THREADS) / THREADS;  // all in flight at once
  uint32_t v[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = static_cast<int>(threadIdx.x) + k * THREADS;
    v[k] = i <= p.grid ? __ldcg(reinterpret_cast<const uint32_t*>(p.errors) + i) : 0u;
  }
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) any |= v[k];
  const bool bad = __syncthreads_or(any != 0);
  if (threadIdx.x < kStatusBytes / 4)
    p.status[threadIdx.x] = !bad ? 0 : (threadIdx.x == 0 ? JFA_ERR_BAD_INPUT : (threadIdx.x == 1 ? kSiteFp8DecodeTable : 0));
}

// Where the parts of an output row lie.
struct F8Row {
  int count;         // parts; 0: the sequence is empty, 1: finished by its part
  bool is_long;
  int step;          // rows from one part to the next
  const float* lse;  // of the first part
  const float* po;
  int64_t out;       // row of O
  int64_t w;         // index of the row's lse among the weights'
  __device__ __forceinline__ F8Row(const Fp8DecodeParams& p, int job, int D) {
    const int hkv = p.c.hkv, G = p.group, nrows = G * p.q_len;
    const int seg = job / nrows, r = job - seg * nrows, b = seg / hkv, h = seg - b * hkv;
    const int base = __ldcg(p.tile_base + b), end = __ldcg(p.tile_base + b + 1);
    const F8Line line(__ldcg(p.tile_base + p.batch), p.max_parts);
    const int i0 = end > base ? line.part_of(base) : 0;
    count = end > base ? line.part_of(end - 1) - i0 + 1 : 0;
    is_long = line.is_long(base, end);
    const int64_t first = ((static_cast<int64_t>(i0) + b) * hkv + h) * nrows + r;
    step = hkv * nrows;
    lse = p.part_lse2 + first;
    po = p.part_o + first * D;
    out = (static_cast<int64_t>(b) * p.q_len + r / G) * p.hq + static_cast<int64_t>(h) * G + r % G;
    w = static_cast<int64_t>(seg) * nrows + r;
  }
};

// The row's lse from its largest part's (0 if every part is empty or NaN) and the sum relative to it.
__device__ __forceinline__ void f8_write_lse(const Fp8DecodeParams& p, const F8Row& row, float top, float z) {
  const float lse2 = z == 0.f ? -INFINITY : top + log2f(z);
  p.lse[row.out] = lse2 * 0.6931471805599453f;
  if (p.w_out) p.lse2[row.w] = f8_weight_lse(lse2);
}

// 32 columns of a row by a block of threads.
template <int D, int THREADS>
__device__ __forceinline__ void join_slice(const Fp8DecodeParams& p, const F8Row& row, int slice) {
  constexpr int kWarps = THREADS / 32, kGroups = THREADS / 8;
  __shared__ float s_f[kFp8MaxWarps];
  __shared__ float s_red[2][kWarps];
  __shared__ float s_o[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = threadIdx.x >> 3, sub = threadIdx.x & 7;
  const int count = row.count, step = row.step;
  const float *lse = row.lse, *po = row.po + 32 * slice;
  auto load = [&](int i) {
    return i < count ? __ldcg(reinterpret_cast<const float4*>(po + static_cast<int64_t>(i) * step * D) + sub)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = load(group + kGroups * k);
  float m = -INFINITY;
  for (int i = threadIdx.x; i < count; i += THREADS) {
    const float y = __ldcg(lse + static_cast<int64_t>(i) * step);
    s_f[i] = y;
    m = fmaxf(m, y);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) s_red[0][warp] = m;
  __syncthreads();
  float top = s_red[0][0];  // the largest lse (0 if every part is empty or NaN)
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_red[0][w]);
  if (top == -INFINITY) top = 0.f;
  float sum = 0.f;
  for (int i = threadIdx.x; i < count; i += THREADS) {
    const float f = ptx::ex2(s_f[i] - top);
    s_f[i] = f;
    sum += f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_red[1][warp] = sum;
  __syncthreads();
  float z = 0.f;  // sum of 2^(lse - top)
#pragma unroll
  for (int w = 0; w < kWarps; ++w) z += s_red[1][w];
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = group; i < count; i += 4 * kGroups) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = i + kGroups * k < count ? s_f[i + kGroups * k] : 0.f;
      o.x += f * v[k].x;
      o.y += f * v[k].y;
      o.z += f * v[k].z;
      o.w += f * v[k].w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load(i + kGroups * (4 + k));
  }
#pragma unroll
  for (int off = 8; off < 32; off <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
  }
  if (lane < 8) *reinterpret_cast<float4*>(&s_o[warp][4 * sub]) = o;
  __syncthreads();
  if (threadIdx.x < 32) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) y += s_o[w][lane];
    p.o[row.out * D + 32 * slice + lane] = __float2bfloat16(z == 0.f ? 0.f : y / z);
    if (lane == 0 && slice == 0) f8_write_lse(p, row, top, z);
  }
}

// A warp per row (`blocks` blocks of four, this one is `block`); the rows of long sequences by slices.
template <int D, int kAtOnce>
__device__ __forceinline__ void join_rows(const Fp8DecodeParams& p, int block, int blocks) {
  constexpr int kPer = D / 32;  // output columns of a lane
  const int lane = threadIdx.x & 31;
  const int seq_rows = p.c.hkv * p.group * p.q_len, rows = p.batch * seq_rows;
  const int mine = block * 4 + static_cast<int>(threadIdx.x >> 5);
  const int many = __ldcg(p.long_list);
  const F8Row row(p, min(mine, rows - 1), D);
  if (mine < rows && row.count != 1 && !row.is_long) {
    auto load = [&](int i, float (&v)[kPer]) {
      const float* src = row.po + static_cast<int64_t>(i) * row.step * D;
      if constexpr (kPer == 4) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src) + lane);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      } else {
        const float2 a = __ldcg(reinterpret_cast<const float2*>(src) + lane);
        v[0] = a.x, v[1] = a.y;
      }
    };
    float v[kAtOnce][kPer], o[kPer];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (k < row.count) load(k, v[k]);
    float y[2];  // lane l: parts l and l + 32
#pragma unroll
    for (int k = 0; k < 2; ++k)
      y[k] = lane + 32 * k < row.count ? __ldcg(row.lse + static_cast<int64_t>(lane + 32 * k) * row.step) : -INFINITY;
    float m = fmaxf(y[0], y[1]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (m == -INFINITY) m = 0.f;
    const float f[2] = {ptx::ex2(y[0] - m), ptx::ex2(y[1] - m)};
    float z = f[0] + f[1];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = 0.f;
    for (int i = 0; i < row.count; i += kAtOnce) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (i + k >= row.count) break;
        const float g = __shfl_sync(0xffffffffu, i < 32 ? f[0] : f[1], i + k);
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] += g * v[k][e];
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (i + kAtOnce + k < row.count) load(i + kAtOnce + k, v[k]);
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    if constexpr (kPer == 4)
      reinterpret_cast<uint2*>(p.o + row.out * D)[lane] =
          make_uint2(ptx::pack_bf16(o[0] * inv, o[1] * inv), ptx::pack_bf16(o[2] * inv, o[3] * inv));
    else
      reinterpret_cast<uint32_t*>(p.o + row.out * D)[lane] = ptx::pack_bf16(o[0] * inv, o[1] * inv);
    if (lane == 0) f8_write_lse(p, row, m, z);
  }
  const int items = seq_rows * (D / 32);
  for (int j = 0; j < many; ++j) {
    const int b = __ldcg(p.long_list + 1 + j);
    for (int item = block; item < items; item += blocks) {
      __syncthreads();  // the last slice is done with
      join_slice<D, 128>(p, F8Row(p, b * seq_rows + item / (D / 32), D), item % (D / 32));
    }
  }
}

constexpr int kF8WideThreads = 256;
template <int D, bool kWide>
__global__ void __launch_bounds__(kWide ? kF8WideThreads : 128) fp8_decode_join_kernel(const Fp8DecodeParams p) {
  wait_prior_grid();
  allow_next_grid();
  if (blockIdx.x == gridDim.x - 1) {
    f8_report<kWide ? kF8WideThreads : 128>(p);
  } else if constexpr (kWide) {
    const F8Row row(p, static_cast<int>(blockIdx.x / (D / 32)), D);
    if (row.count != 1) join_slice<D, kF8WideThreads>(p, row, static_cast<int>(blockIdx.x % (D / 32)));
  } else {
    join_rows<D, 16>(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x) - 1);
  }
}

// The rows' lse of a sequence and head, joined from its parts once more (the join's own may not be
// there yet): lane r + kRows j reads row r's parts j, j + 32 / kRows, ...
template <int kRows>
__device__ __forceinline__ void f8_join_lse(const Fp8DecodeParams& p, int b, int h, float (&z)[kRows]) {
  const int lane = threadIdx.x & 31, hkv = p.c.hkv, nrows = p.group * p.q_len, r = lane % kRows;
  const F8Line line(p.tile_base[p.batch], p.max_parts);
  const int i0 = line.part_of(p.tile_base[b]), count = line.part_of(p.tile_base[b + 1] - 1) - i0 + 1;
  float y = INFINITY;
  if (count == 1) {  // its part has finished it
    if (r < nrows) y = __ldcg(p.lse2 + (static_cast<int64_t>(b) * hkv + h) * nrows + r);
  } else {
    const float* lse = p.part_lse2 + ((static_cast<int64_t>(i0) + b) * hkv + h) * nrows + r;
    const int64_t step = static_cast<int64_t>(hkv) * nrows;
    constexpr int kStride = 32 / kRows, kLoads = kRows < 4 ? kRows : 4;  // parts a round: kStride * kLoads
    float m = kF8NoRef, sum = 0.f;
    for (int i = lane / kRows; i < count; i += kStride * kLoads) {
      float x[kLoads], top = m;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        x[k] = i + k * kStride < count && r < nrows ? __ldcg(lse + (i + k * kStride) * step) : -INFINITY;
        top = fmaxf(top, x[k]);
      }
      sum *= ptx::ex2(m - top);
      m = top;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) sum += ptx::ex2(x[k] - m);
    }
#pragma unroll
    for (int off = kRows; off < 32; off <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off), top = fmaxf(m, m2);
      const float s2 = __shfl_xor_sync(0xffffffffu, sum, off);
      sum = sum * ptx::ex2(m - top) + s2 * ptx::ex2(m2 - top);
      m = top;
    }
    y = sum == 0.f ? INFINITY : m + log2f(sum);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) z[k] = __shfl_sync(0xffffffffu, y, k);
}

// w_out = decay * w_in + sum over the rows of 2^(score - lse). Like the main kernel a
// warp takes a part of the line of tiles for one head: a lane per token, two tiles
// at a time, the rows' lse in registers, kAhead pairs of tiles and kRows rows
// (16 loads a lane) in flight. Bound by HBM: 4 bytes per row and 8 per token and head.
template <int kAhead, int kRows, bool kJoined>
__device__ __forceinline__ void add_weights(const Fp8DecodeParams& p, int max_parts, int first, int stride) {
  const int lane = threadIdx.x & 31;
  const int hkv = p.c.hkv, nrows = p.group * p.q_len;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const F8Line line(p.tile_base[p.batch], max_parts);
  const int jobs = static_cast<int>(line.parts) * hkv;
  const int64_t pair = static_cast<int64_t>(hkv) * nrows * 32;  // scores from one pair of tiles to the next
  for (int job = first; job < jobs; job += stride) {
    const int part = fast_div(job, p.by_heads), h = job - part * hkv;
    int x = line.begin(part);
    const int x1 = line.begin(part + 1);
    int b = f8_find_sequence(p.tile_base, p.batch, x, 0);
    while (x < x1) {
      if (p.tile_base[b + 1] <= x) b = f8_next_sequence(p.tile_base, p.batch, x, b);
      bool bad;
      const int base = p.tile_base[b], stop = min(p.tile_base[b + 1], x1);
      const int L = f8_length(p, b, &bad), end = min(L, (stop - base) * 16);  // tokens of this part of the sequence
      const int64_t seg = static_cast<int64_t>(b) * hkv + h;
      float z[kRows];
      if constexpr (kJoined) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) z[r] = r < nrows ? p.lse2[seg * nrows + r] : INFINITY;
      } else {
        f8_join_lse<kRows>(p, b, h, z);
      }
      int t = (x - base) * 16 + lane;
      const float* s = p.scores + ((static_cast<int64_t>(x) + (lane >> 4)) * hkv + h) * nrows * 16 + (lane & 15);
      const float* in = p.w_in ? p.w_in + seg * cap : nullptr;
      float* out = p.w_out + seg * cap;
      for (; t - lane < end; t += 32 * kAhead, s += kAhead * pair) {
        float v[kAhead][kRows], sum[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const bool have = t + 32 * k < end;
          sum[k] = have && in ? in[t + 32 * k] : 0.f;
#pragma unroll
          for (int r = 0; r < kRows; ++r) v[k][r] = have && r < nrows ? s[k * pair + r * 16] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          sum[k] *= p.decay;
          float all = sum[k];
#pragma unroll
          for (int r = 0; r < kRows; ++r) all += ptx::ex2(v[k][r] - z[r]);
          // The first `hidden` rows do not see this token: they add nothing, a NaN lse of theirs neither.
          // (A branch that few warps take: with a test of every row the loads no longer go out together,
          // 36 against 41 us for 87 x 2k-8k tokens of one KV head, 8 rows, behind the join.)
          const int newer = t + 32 * k - (L - p.q_len);
          if (newer > 0) {
            const int hidden = newer * p.group;
            all = sum[k];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
              if (r >= hidden) all += ptx::ex2(v[k][r] - z[r]);
          }
          sum[k] = all;
          if (t + 32 * k < end) out[t + 32 * k] = sum[k];
        }
      }
      x = stop;
    }
  }
}

// The weights by themselves, behind the join.
constexpr int kF8WeightWarps = 8;
template <int kAhead, int kRows>
__global__ void __launch_bounds__(32 * kF8WeightWarps) fp8_decode_weights_kernel(const Fp8DecodeParams p, int max_parts) {
  wait_prior_grid();
  add_weights<kAhead, kRows, true>(p, max_parts, blockIdx.x * kF8WeightWarps + (threadIdx.x >> 5),
                                   gridDim.x * kF8WeightWarps);
}

// The weights beside the join of a warp per row: the first `blocks` blocks add weights, the others join
// rows, the last one reports. One launch less, and neither waits for the other: 32 x 1k-32k tokens 206.4 ->
// 204.8 us, 24 x 37-4k of head_dim 64 21.3 -> 19.3, and 3 us less on the host.
template <int D, int kAhead, int kRows>
__global__ void __launch_bounds__(128) fp8_decode_finish_kernel(const Fp8DecodeParams p, int max_parts, int blocks) {
  wait_prior_grid();
  const int block = static_cast<int>(blockIdx.x);
  if (block < blocks)
    add_weights<kAhead, kRows, false>(p, max_parts, block * 4 + (threadIdx.x >> 5), blocks * 4);
  else if (blockIdx.x == gridDim.x - 1)
    f8_report<128>(p);
  else
    join_rows<D, 8>(p, block - blocks, static_cast<int>(gridDim.x) - 1 - blocks);
}

// ------------------------------------------------------------------ launchers

template <int D, int NR, bool W>
static cudaError_t launch_main(const Fp8DecodeParams& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  using T = F8Tile<D, NR>;
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(fp8_decode_kernel<D, NR, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                T::kRingBytes);
  });
  if (e != cudaSuccess) return e;
  if (p.batch > kF8ScanBatch)
    return launch_after(fp8_decode_kernel<D, NR, W>, dim3(grid), dim3(32 * kF8Warps), T::kRingBytes, stream, p);
  fp8_decode_kernel<D, NR, W><<<grid, 32 * kF8Warps, T::kRingBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_dim(Fp8DecodeParams& p, void* events, int sms, cudaStream_t stream) {
  const int nrows = p.group * p.q_len;
  const bool w = p.w_out != nullptr;
  const int per_sm = nrows <= 8 ? F8Tile<D, 1>::kCtasPerSm : F8Tile<D, 2>::kCtasPerSm;
  const int64_t tiles = static_cast<int64_t>(p.batch) * fp8_seq_tiles(p.max_pages, p.page_size);
  // every resident warp gets one part of one head
  const int warps = std::min(sms * per_sm * kF8Warps, kFp8MaxWarps);
  p.max_parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(warps / p.c.hkv, tiles)));
  const int grid = static_cast<int>(
      std::min<int64_t>(warps / kF8Warps, (static_cast<int64_t>(p.max_parts) * p.c.hkv + kF8Warps - 1) / kF8Warps));
  p.grid = grid;
  p.by_heads = make_fast_div(p.c.hkv);
  cudaError_t e;
  if (p.batch > kF8ScanBatch) {
    fp8_decode_plan_kernel<<<1, 1024, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaEvent_t* ev = static_cast<cudaEvent_t*>(events);
  if (ev) cudaEventRecord(ev[0], stream);
  if (nrows <= 8)
    e = w ? launch_main<D, 1, true>(p, grid, stream) : launch_main<D, 1, false>(p, grid, stream);
  else
    e = w ? launch_main<D, 2, true>(p, grid, stream) : launch_main<D, 2, false>(p, grid, stream);
  if (ev) cudaEventRecord(ev[1], stream);
  if (e != cudaSuccess) return e;
  // The wide join past 32 parts a sequence on average, half of what a warp joins: lengths differ. With
  // 25 parts, 24 x 37-4k tokens of head_dim 64 take 26 us by it and 21 by rows; with 6 to 28 parts, 8 KV heads,
  // 51 x 10k 185 and 154, 11 x 32k 121 and 114. With 34 to 61 parts even lengths would take less by rows
  // still (9 x 8k 37 and 32, 5 x 8k 25 and 24), mixed ones more: 5 x 1k-32k 37 and 50, 41 x 1k-32k of one KV
  // head 42 and 82, one of 131k with four of 500 52 and 62. With 101 parts 3 x 32k take 39 and 76.
  const uint32_t rows = static_cast<uint32_t>(p.batch) * p.c.hkv * nrows, join_blocks = (rows + 3) / 4 + 1;
  const bool wide = p.max_parts > 32 * p.batch;
  auto join = [&] {
    return wide ? launch_after(fp8_decode_join_kernel<D, true>, dim3(rows * (D / 32) + 1), dim3(kF8WideThreads), 0, stream, p)
                : launch_after(fp8_decode_join_kernel<D, false>, dim3(join_blocks), dim3(128), 0, stream, p);
  };
  if (!w) return join();
  // The weights beside the join read the lse of a sequence's parts again in every warp: not where there can
  // be thousands. Even lengths take less beside it whatever the parts (11 to 87 x 2k-8k 32 us against 34, and
  // 3 less on the host), one sequence of 65k among 500s more: with 304 parts 48 against 44 (4 rows), 53
  // against 42 (16 rows, 4 KV heads), with 608 39 against 32 and 66 against 32, with 1216 36 against 30 and
  // 96 against 32.
  const bool beside = !wide && p.max_parts <= 640;
  const int weight_warps = beside ? sms * 5 * 4 : sms * 4 * kF8WeightWarps;
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(weight_warps / p.c.hkv, tiles)));
  if (beside) {
    const int blocks = weight_warps / 4;  // five of the six or seven blocks that fit an SM: the join runs beside them
    const dim3 g(blocks + join_blocks), block(128);
    if (nrows <= 4) return launch_after(fp8_decode_finish_kernel<D, 4, 4>, g, block, 0, stream, p, parts, blocks);
    if (nrows <= 8) return launch_after(fp8_decode_finish_kernel<D, 2, 8>, g, block, 0, stream, p, parts, blocks);
    return launch_after(fp8_decode_finish_kernel<D, 1, 16>, g, block, 0, stream, p, parts, blocks);
  }
  e = join();
  if (e != cudaSuccess) return e;
  const dim3 g(sms * 4), block(32 * kF8WeightWarps);
  if (nrows <= 4) return launch_after(fp8_decode_weights_kernel<4, 4>, g, block, 0, stream, p, parts);
  if (nrows <= 8) return launch_after(fp8_decode_weights_kernel<2, 8>, g, block, 0, stream, p, parts);
  return launch_after(fp8_decode_weights_kernel<1, 16>, g, block, 0, stream, p, parts);
}

cudaError_t launch_decode_fp8(const jfa_decode_fp8_args& a, const Fp8DecodeBuffers& w, int sms, cudaStream_t stream) {
  Fp8DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.c.kc = static_cast<uint8_t*>(const_cast<void*>(a.k_cache));
  p.c.vc = static_cast<uint8_t*>(const_cast<void*>(a.v_cache));
  p.c.ks = const_cast<float*>(a.k_scale);
  p.c.vs = const_cast<float*>(a.v_scale);
  p.c.hkv = a.kv_heads;
  p.c.num_pages = a.num_pages;
  p.c.block_shift = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.c.page = make_fast_div(a.page_size);
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.batch = a.batch;
  p.hq = a.q_heads;
  p.group = a.q_heads / a.kv_heads;
  p.q_len = a.q_len;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.tile_base = w.tile_base;
  p.long_list = w.long_list;
  p.errors = w.errors;
  p.part_o = w.part_o;
  p.part_lse2 = w.part_lse2;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.lse2 = w.lse2;
  p.scores = w.scores;
  p.w_in = a.weights;
  p.w_out = a.weights_out;
  p.decay = a.weights ? a.decay : 0.f;
  p.status = w.status;
  return a.head_dim == 128 ? launch_dim<128>(p, a.main_kernel_events, sms, stream)
                           : launch_dim<64>(p, a.main_kernel_events, sms, stream);
}

}  // namespace jfa
