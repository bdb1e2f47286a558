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
//  * Every lane copies the 16-byte pieces it will read itself with cp.async
//    into a per-warp ring (a piece of 32 lanes is 512 contiguous bytes), so
//    the ring needs no synchronisation beyond the warp's own.
//  * Work is split evenly over all CTAs, whatever the lengths: the 16-token
//    tiles of all (sequence, KV head) segments form one line that is cut into
//    equal parts. A segment inside one part is finished there; one that was
//    cut leaves a partial result per part, joined by a second kernel in the
//    order of the parts (no atomics on results: the outcome depends on the
//    lengths and the SM count only).
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
#include <cuda_fp16.h>

#include "fp8_cache.cuh"

namespace jfa {

struct Fp8DecodeParams {
  const __nv_bfloat16* q;
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  int32_t batch, hq, group, q_len, max_pages, page_size;
  float scale_log2;
  int32_t* lens;       // [B] checked lengths
  int32_t* tile_base;  // [B + 1] 16-token tiles of the sequences before b
  int32_t parts;       // CTAs of the main kernel
  float* part_o;       // [parts + B * hkv][rows][D], normalised
  float* part_lse2;    // [parts + B * hkv][rows], log2, -inf when empty
  __nv_bfloat16* o;
  float* lse;          // [B, q_len, Hq] natural log
  float* lse2;         // [B, hkv, rows] log2 (weights only)
  float* scores;       // [tiles][rows][16] log2 units (weights only)
  const float* w_in;   // [B, hkv, max_pages * page_size] or null
  float* w_out;
  float decay;
  int32_t* status;
};

constexpr int kF8Warps = 4;
constexpr int kF8Stages = 4;
constexpr int kF8CtasPerSm = 3;
constexpr int kF8MinTiles = 8;  // fewest tiles of a part (two per warp)
// A score may pass its reference by this much before the reference moves.
constexpr float kF8Slack = 8.f;
// w's reference lies this far below the largest s + log2 vs when it is set.
constexpr float kF8WShift = 7.f;
constexpr float kF8NoRef = -3.0e38f;  // a reference before the first visible token

template <int D>
struct F8Tile {
  static constexpr int kKPieces = 2 * (D / 64);  // 16-byte pieces of K a lane copies per tile
  static constexpr int kVBytes = D / 8;          // bytes of a V piece (16 or 8)
  static constexpr int kVOff = kKPieces * 512;
  static constexpr int kScaleOff = kVOff + 4 * 32 * kVBytes;
  static constexpr int kStageBytes = kScaleOff + 128;
  static constexpr int kRingBytes = kF8Warps * kF8Stages * kStageBytes;
};

__device__ __forceinline__ void f8_cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void f8_cp_async8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// 8 x 8 matrix of 16-bit elements, transposed between the lanes of a warp.
__device__ __forceinline__ uint32_t f8_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One block: clears the status block, checks the lengths and numbers the tiles.
__global__ void __launch_bounds__(1024) fp8_decode_plan_kernel(const Fp8DecodeParams p) {
  allow_next_grid();
  __shared__ int32_t warp_sum[32];
  __shared__ int32_t running;
  if (threadIdx.x < kStatusBytes / 4) p.status[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    running = 0;
    p.tile_base[0] = 0;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < p.batch) {
      int L = p.seqlens[b];
      if (L < 0 || L > cap || (L > 0 && p.c.num_pages == 0)) {
        flag_bad_cache(p.status, kSiteFp8DecodeTable);
        L = 0;
      }
      p.lens[b] = L;
      n = (L + 15) >> 4;
    }
    int x = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int s = warp_sum[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    const int before = running + (warp > 0 ? warp_sum[warp - 1] : 0);
    if (b < p.batch) p.tile_base[b + 1] = before + x;
    __syncthreads();
    if (threadIdx.x == 0) running += warp_sum[31];
    __syncthreads();
  }
}

// The line of tiles, cut into parts of equal length.
struct F8Line {
  int64_t total;  // tiles of all segments
  int64_t parts;  // parts in use
  __device__ __forceinline__ F8Line(const int32_t* tile_base, int batch, int hkv, int max_parts) {
    total = static_cast<int64_t>(tile_base[batch]) * hkv;
    parts = min(static_cast<int64_t>(max_parts), (total + kF8MinTiles - 1) / kF8MinTiles);
  }
  __device__ __forceinline__ int64_t begin(int64_t i) const { return parts ? i * total / parts : 0; }
  // the part that holds tile x: the last i with floor(i total / parts) <= x
  __device__ __forceinline__ int64_t part_of(int64_t x) const { return ((x + 1) * parts - 1) / total; }
};

// The sequence whose tiles hold tile x of the line (a warp's lanes look at 32 bounds at a time).
__device__ __forceinline__ int f8_find_sequence(const int32_t* tile_base, int batch, int hkv, int64_t x) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < batch; b0 += 32) {
    const int b = b0 + lane;
    const bool past = b < batch && static_cast<int64_t>(tile_base[b + 1]) * hkv > x;
    const uint32_t m = __ballot_sync(0xffffffffu, past);
    if (m) return b0 + __ffs(m) - 1;
  }
  return batch - 1;
}

template <int D, int NR, bool WEIGHTS>
__global__ void __launch_bounds__(128, kF8CtasPerSm) fp8_decode_kernel(const Fp8DecodeParams p) {
  using T = F8Tile<D>;
  constexpr int kSteps = D / 16;   // MMA steps of Q K^T, and of P V
  constexpr int kEpl = D / 8;      // head dimensions a lane holds of each of its query rows
  constexpr int kRows = 8 * NR;
  constexpr int kRowStride = D + 4;  // padded: the partials' rows start on different banks
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_m[kF8Warps][kRows], s_n[kF8Warps][kRows], s_l[kF8Warps][kRows];
  static_assert(kF8Warps * kRows * kRowStride * 4 <= T::kRingBytes, "the partials reuse the ring");
  float* s_o = reinterpret_cast<float*>(smem);

  wait_prior_grid();  // the plan (lengths, tile numbers, cleared status)
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, qq = lane & 3;
  const int hkv = p.c.hkv, G = p.group, QL = p.q_len, nrows = G * QL;
  const F8Line line(p.tile_base, p.batch, hkv, p.parts);
  if (blockIdx.x >= line.parts) return;
  int64_t x = line.begin(blockIdx.x);
  const int64_t x_end = line.begin(blockIdx.x + 1);
  int b = f8_find_sequence(p.tile_base, p.batch, hkv, x);
  uint8_t* ring = smem + warp * kF8Stages * T::kStageBytes;
  const uint32_t ring_u32 = ptx::smem_u32(ring);
  const int64_t token_stride = static_cast<int64_t>(hkv) * D;

  while (x < x_end) {
    // ---- the segment (sequence b, KV head h) and this part's tiles of it
    while (static_cast<int64_t>(p.tile_base[b + 1]) * hkv <= x) ++b;
    const int64_t seq0 = static_cast<int64_t>(p.tile_base[b]) * hkv;
    const int ntiles = p.tile_base[b + 1] - p.tile_base[b];
    const int h = static_cast<int>((x - seq0) / ntiles);
    const int64_t seg0 = seq0 + static_cast<int64_t>(h) * ntiles;
    const int t_lo = static_cast<int>(x - seg0);
    const int t_hi = static_cast<int>(min(static_cast<int64_t>(ntiles), x_end - seg0));
    const int L = p.lens[b];
    const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    const int nmine = (t_hi - t_lo - warp + kF8Warps - 1) / kF8Warps;  // may be <= 0

    // ---- page of this lane's token (lane % 16) of the warp's tile i
    auto page_entry = [&](int i) -> int {
      const int tok = (t_lo + warp + kF8Warps * i) * 16 + (lane & 15);
      return (i < nmine && tok < L) ? pt[fast_div(tok, p.c.page)] : 0;
    };
    auto issue = [&](int i, int page) {
      if (i < nmine) {
        const int t0 = (t_lo + warp + kF8Warps * i) * 16;
        const int tok = t0 + (lane & 15);
        const bool in = tok < L;
        if (in && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.num_pages)) {
          flag_bad_cache(p.status, kSiteFp8DecodeTable);
          page = 0;
        }
        const int slot = tok - fast_div(tok, p.c.page) * p.page_size;
        const int row = in ? page * p.page_size + slot : 0;
        const uint32_t st = ring_u32 + (i % kF8Stages) * T::kStageBytes;
        const int64_t sc = static_cast<int64_t>(row >> p.c.block_shift) * hkv + h;
        f8_cp_async4(st + T::kScaleOff + lane * 4, (lane < 16 ? p.c.ks : p.c.vs) + sc, in ? 4 : 0);
        const uint8_t* kb = p.c.kc + static_cast<int64_t>(h) * D + 16 * qq;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = __shfl_sync(0xffffffffu, row, gq + 8 * u);
          const uint32_t n = t0 + gq + 8 * u < L ? 16 : 0;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            f8_cp_async16(st + ((u * (D / 64) + c) * 32 + lane) * 16, kb + r * token_stride + 64 * c, n);
        }
        const uint8_t* vb = p.c.vc + static_cast<int64_t>(h) * D + T::kVBytes * gq;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int tk = 2 * qq + (w & 1) + 8 * (w >> 1);
          const int r = __shfl_sync(0xffffffffu, row, tk);
          const bool ok = t0 + tk < L;
          const uint32_t dst = st + T::kVOff + (w * 32 + lane) * T::kVBytes;
          if constexpr (D == 128)
            f8_cp_async16(dst, vb + r * token_stride, ok ? 16 : 0);
          else
            f8_cp_async8(dst, vb + r * token_stride, ok ? 8 : 0);
        }
      }
      f8_commit();  // one group per call, empty past the last tile
    };
    {
      int pg[kF8Stages - 1];
#pragma unroll
      for (int i = 0; i < kF8Stages - 1; ++i) pg[i] = page_entry(i);
#pragma unroll
      for (int i = 0; i < kF8Stages - 1; ++i) issue(i, pg[i]);
    }
    int pg_next = page_entry(kF8Stages - 1);

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
            // bytes 4 w .. of the 16: element 8 e + 2 k is step w = 2 e + k / 2, register k % 2
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

    for (int i = 0; i < nmine; ++i) {
      const int tile = t_lo + warp + kF8Warps * i;
      const int t0 = tile * 16;
      __syncwarp();  // every lane has read the slot that is refilled now (tile i - 1)
      issue(i + kF8Stages - 1, pg_next);
      pg_next = page_entry(i + kF8Stages);
      f8_wait<kF8Stages - 1>();  // tile i has landed
      __syncwarp();              // the scales come from other lanes' copies
      const uint8_t* st = ring + (i % kF8Stages) * T::kStageBytes;
      const float* sc = reinterpret_cast<const float*>(st + T::kScaleOff);
      const float ks0 = sc[gq], ks1 = sc[gq + 8];
      const float lv0 = __log2f(sc[16 + gq]), lv1 = __log2f(sc[24 + gq]);

      // S^T = K Q^T
      float s[NR][4];
#pragma unroll
      for (int u = 0; u < NR; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(st + (c * 32 + lane) * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(st + ((D / 64 + c) * 32 + lane) * 16);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16(w0[w], a0, a2);
          e4m3x4_to_f16(w1[w], a1, a3);
#pragma unroll
          for (int u = 0; u < NR; ++u) f8_mma(s[u], a0, a1, a2, a3, qb[u][4 * c + w][0], qb[u][4 * c + w][1]);
        }
      }
      // scaled scores: s[u][0..1] token g, rows 2q and 2q + 1; s[u][2..3] token g + 8
      const bool partial = t0 + 16 > lim_min;
      bool raise = false;
#pragma unroll
      for (int u = 0; u < NR; ++u) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[u][e] *= ks0 * rq[u][e];
          s[u][2 + e] *= ks1 * rq[u][e];
          if (partial) {
            if (t0 + gq >= lim[u][e]) s[u][e] = -INFINITY;
            if (t0 + gq + 8 >= lim[u][e]) s[u][2 + e] = -INFINITY;
          }
          raise |= fmaxf(s[u][e], s[u][2 + e]) > m[u][e] + kF8Slack;
          raise |= fmaxf(s[u][e] + lv0, s[u][2 + e] + lv1) > n[u][e] + (kF8WShift + kF8Slack);
        }
      }
      if constexpr (WEIGHTS) {
        float* out = p.scores + (seg0 + tile) * static_cast<int64_t>(nrows) * 16;
#pragma unroll
        for (int u = 0; u < NR; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * u + 2 * qq + e;
            if (r < nrows) {
              out[r * 16 + gq] = s[u][e];
              out[r * 16 + gq + 8] = s[u][2 + e];
            }
          }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int u = 0; u < NR; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = fmaxf(s[u][e], s[u][2 + e]);
            float c = fmaxf(s[u][e] + lv0, s[u][2 + e] + lv1);
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
      uint32_t pb[NR][2];
#pragma unroll
      for (int u = 0; u < NR; ++u) {
#pragma unroll
        for (int e = 0; e < 2; ++e) l[u][e] += ptx::ex2(s[u][e] - m[u][e]) + ptx::ex2(s[u][2 + e] - m[u][e]);
        pb[u][0] = f8_transpose(f8_pack_f16(ptx::ex2(s[u][0] + lv0 - n[u][0]), ptx::ex2(s[u][1] + lv0 - n[u][1])));
        pb[u][1] = f8_transpose(f8_pack_f16(ptx::ex2(s[u][2] + lv1 - n[u][0]), ptx::ex2(s[u][3] + lv1 - n[u][1])));
      }
      // O^T += V^T P^T
      uint32_t vw[4][kEpl / 4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint8_t* src = st + T::kVOff + (w * 32 + lane) * T::kVBytes;
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(src);
          vw[w][0] = v.x;
          vw[w][1] = v.y;
          vw[w][2] = v.z;
          vw[w][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          vw[w][0] = v.x;
          vw[w][1] = v.y;
        }
      }
      if (partial && QL > 1) {
        // A value that some rows may not see must not reach them even as
        // 0 * NaN: NaN codes leave V and are put into the rows that do see
        // them, where a second product counts them.
        bool bad = false;
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int k = 0; k < kEpl / 4; ++k) bad |= e4m3_any_nan(vw[w][k]);
        if (__any_sync(0xffffffffu, bad)) {
          uint32_t one[4][kEpl / 4];  // e4m3 1.0 (0x38) where the code is NaN
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int k = 0; k < kEpl / 4; ++k) {
              const uint32_t hit = (((vw[w][k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;  // 0x01 per byte
              one[w][k] = hit * 0x38u;
              vw[w][k] &= ~(hit * 0xFFu);
            }
#pragma unroll
          for (int u = 0; u < NR; ++u) {
            float see[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              see[e] = t0 + gq < lim[u][e] ? 1.f : 0.f;
              see[2 + e] = t0 + gq + 8 < lim[u][e] ? 1.f : 0.f;
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
      for (int j = 0; j < kSteps; ++j) {
        // bytes (token a, d), (token a + 1, d), (token a, d + 1), (token a + 1, d + 1)
        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16(__byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel), a0, a1);
        e4m3x4_to_f16(__byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel), a2, a3);
#pragma unroll
        for (int u = 0; u < NR; ++u) f8_mma(acc[u][j], a0, a1, a2, a3, pb[u][0], pb[u][1]);
      }
    }

    // ---- join the four warps
    f8_wait<0>();
    __syncthreads();  // every warp is done with the ring before it holds the partials
#pragma unroll
    for (int u = 0; u < NR; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[u][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int r = 8 * u + 2 * qq + e;
        if (gq == 0) {
          s_m[warp][r] = m[u][e];
          s_n[warp][r] = n[u][e];
          s_l[warp][r] = sum;
        }
        float* dst = s_o + (warp * kRows + r) * kRowStride + kEpl * gq;
#pragma unroll
        for (int j = 0; j < kSteps; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) =
              make_float4(acc[u][j][e], acc[u][j][2 + e], acc[u][j + 1][e], acc[u][j + 1][2 + e]);
      }
    __syncthreads();
    const int seg = b * hkv + h;
    const bool whole = t_lo == 0 && t_hi == ntiles;
    for (int idx = threadIdx.x; idx < nrows * (D / 4); idx += 128) {
      const int r = idx / (D / 4), c4 = (idx % (D / 4)) * 4;
      float M = s_m[0][r];
#pragma unroll
      for (int w = 1; w < kF8Warps; ++w) M = fmaxf(M, s_m[w][r]);
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kF8Warps; ++w) {
        sum += s_l[w][r] * ptx::ex2(s_m[w][r] - M);
        const float f = ptx::ex2(s_n[w][r] - M);
        const float4 a = *reinterpret_cast<const float4*>(s_o + (w * kRows + r) * kRowStride + c4);
        v.x += a.x * f;
        v.y += a.y * f;
        v.z += a.z * f;
        v.w += a.w * f;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw no token: zeros (NaN stays NaN)
      v.x *= inv;
      v.y *= inv;
      v.z *= inv;
      v.w *= inv;
      const float z = sum == 0.f ? -INFINITY : M + log2f(sum);
      if (whole) {
        const int64_t row = (static_cast<int64_t>(b) * QL + r / G) * p.hq + static_cast<int64_t>(h) * G + r % G;
        *reinterpret_cast<uint2*>(p.o + row * D + c4) = make_uint2(ptx::pack_bf16(v.x, v.y), ptx::pack_bf16(v.z, v.w));
        if (c4 == 0) {
          p.lse[row] = z * 0.6931471805599453f;
          if (WEIGHTS) p.lse2[static_cast<int64_t>(seg) * nrows + r] = z;
        }
      } else {
        const int64_t row = (static_cast<int64_t>(blockIdx.x) + seg) * nrows + r;
        *reinterpret_cast<float4*>(p.part_o + row * D + c4) = v;
        if (c4 == 0) p.part_lse2[row] = z;
      }
    }
    __syncthreads();  // the ring is filled again for the next segment
    x = seg0 + t_hi;
  }
}

// Joins the parts of the segments that were cut (one warp per output row):
// lse = log2 sum_i 2^lse_i, O = sum_i 2^(lse_i - lse) O_i, in the order of the
// parts; a sequence without tokens gets zeros and -inf.
template <int D>
__global__ void __launch_bounds__(128) fp8_decode_join_kernel(const Fp8DecodeParams p, int weights) {
  wait_prior_grid();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hkv = p.c.hkv, G = p.group, nrows = G * p.q_len;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * 4 + warp;  // (segment, row)
  if (job >= static_cast<int64_t>(p.batch) * hkv * nrows) return;
  const int seg = static_cast<int>(job / nrows), r = static_cast<int>(job % nrows);
  const int b = seg / hkv, h = seg % hkv;
  const F8Line line(p.tile_base, p.batch, hkv, p.parts);
  const int ntiles = p.tile_base[b + 1] - p.tile_base[b];
  const int64_t row = (static_cast<int64_t>(b) * p.q_len + r / G) * p.hq + static_cast<int64_t>(h) * G + r % G;
  constexpr int kPer = D / 32;  // output columns of a lane
  float o[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = 0.f;
  float z = -INFINITY;
  if (ntiles > 0) {
    const int64_t x0 = static_cast<int64_t>(p.tile_base[b]) * hkv + static_cast<int64_t>(h) * ntiles;
    const int64_t i0 = line.part_of(x0), i1 = line.part_of(x0 + ntiles - 1);
    if (i0 == i1) return;  // finished by its part
    float M = -INFINITY;
    bool nan = false;
    for (int64_t i = i0 + lane; i <= i1; i += 32) {
      const float y = __ldcg(p.part_lse2 + (i + seg) * nrows + r);
      nan |= y != y;
      M = fmaxf(M, y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __any_sync(0xffffffffu, nan);
    float Z = 0.f;
    if (M != -INFINITY || nan) {
      const float base = M == -INFINITY ? 0.f : M;
      for (int64_t i = i0; i <= i1; i += 8) {
        float f[8], v[8][kPer];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool in = i + k <= i1;
          const int64_t pr = (min(i + k, i1) + seg) * nrows + r;
          f[k] = in ? ptx::ex2(__ldcg(p.part_lse2 + pr) - base) : 0.f;
          if constexpr (kPer == 4) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(p.part_o + pr * D) + lane);
            v[k][0] = a.x, v[k][1] = a.y, v[k][2] = a.z, v[k][3] = a.w;
          } else {
            const float2 a = __ldcg(reinterpret_cast<const float2*>(p.part_o + pr * D) + lane);
            v[k][0] = a.x, v[k][1] = a.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (i + k > i1) break;
          Z += f[k];
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[e] += f[k] * v[k][e];
        }
      }
      const float inv = 1.f / Z;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] *= inv;
      z = base + log2f(Z);
    }
  }
  if constexpr (kPer == 4)
    reinterpret_cast<uint2*>(p.o + row * D)[lane] = make_uint2(ptx::pack_bf16(o[0], o[1]), ptx::pack_bf16(o[2], o[3]));
  else
    reinterpret_cast<uint32_t*>(p.o + row * D)[lane] = ptx::pack_bf16(o[0], o[1]);
  if (lane == 0) {
    p.lse[row] = z * 0.6931471805599453f;
    if (weights) p.lse2[static_cast<int64_t>(seg) * nrows + r] = z;
  }
}

// w_out = decay * w_in + sum over the rows of 2^(score - lse): half a warp per
// tile, one lane per token; the blocks share the line of tiles evenly.
__global__ void __launch_bounds__(256) fp8_decode_weights_kernel(const Fp8DecodeParams p) {
  wait_prior_grid();
  const int hkv = p.c.hkv, nrows = p.group * p.q_len;
  const int64_t total = static_cast<int64_t>(p.tile_base[p.batch]) * hkv;
  int64_t x = static_cast<int64_t>(blockIdx.x) * total / gridDim.x;
  const int64_t x_end = static_cast<int64_t>(blockIdx.x + 1) * total / gridDim.x;
  if (x >= x_end) return;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  int b = f8_find_sequence(p.tile_base, p.batch, hkv, x);
  const int half = threadIdx.x >> 4, tk = threadIdx.x & 15;
  while (x < x_end) {
    while (static_cast<int64_t>(p.tile_base[b + 1]) * hkv <= x) ++b;
    const int64_t seq0 = static_cast<int64_t>(p.tile_base[b]) * hkv;
    const int ntiles = p.tile_base[b + 1] - p.tile_base[b];
    const int h = static_cast<int>((x - seq0) / ntiles);
    const int64_t seg0 = seq0 + static_cast<int64_t>(h) * ntiles;
    const int t_hi = static_cast<int>(min(static_cast<int64_t>(ntiles), x_end - seg0));
    const int64_t seg = static_cast<int64_t>(b) * hkv + h;
    const int L = p.lens[b];
    const float* lse2 = p.lse2 + seg * nrows;
    for (int tile = static_cast<int>(x - seg0) + half; tile < t_hi; tile += 16) {
      const int t = tile * 16 + tk;
      if (t >= L) continue;
      const float* s = p.scores + (seg0 + tile) * nrows * 16 + tk;
      float sum = 0.f;
      for (int r = 0; r < nrows; ++r) {
        const float z = lse2[r];
        sum += z == -INFINITY ? 0.f : ptx::ex2(s[r * 16] - z);
      }
      const int64_t at = seg * cap + t;
      p.w_out[at] = p.w_in ? fmaf(p.decay, p.w_in[at], sum) : sum;
    }
    x = seg0 + t_hi;
  }
}

// ------------------------------------------------------------------ launchers

int fp8_decode_parts(int sms) { return sms * kF8CtasPerSm; }

template <int D, int NR, bool W>
static cudaError_t launch_main(const Fp8DecodeParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(fp8_decode_kernel<D, NR, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                F8Tile<D>::kRingBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_after(fp8_decode_kernel<D, NR, W>, dim3(p.parts), dim3(128), F8Tile<D>::kRingBytes, stream, p);
}

template <int D>
static cudaError_t launch_dim(const Fp8DecodeParams& p, void* events, int sms, cudaStream_t stream) {
  const int nrows = p.group * p.q_len;
  const bool w = p.w_out != nullptr;
  fp8_decode_plan_kernel<<<1, 1024, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaEvent_t* ev = static_cast<cudaEvent_t*>(events);
  if (ev) cudaEventRecord(ev[0], stream);
  if (nrows <= 8)
    e = w ? launch_main<D, 1, true>(p, stream) : launch_main<D, 1, false>(p, stream);
  else
    e = w ? launch_main<D, 2, true>(p, stream) : launch_main<D, 2, false>(p, stream);
  if (ev) cudaEventRecord(ev[1], stream);
  if (e != cudaSuccess) return e;
  const int64_t jobs = static_cast<int64_t>(p.batch) * p.c.hkv * nrows;
  e = launch_after(fp8_decode_join_kernel<D>, dim3(static_cast<uint32_t>((jobs + 3) / 4)), dim3(128), 0, stream, p,
                   w ? 1 : 0);
  if (e != cudaSuccess || !w) return e;
  return launch_after(fp8_decode_weights_kernel, dim3(static_cast<uint32_t>(sms * 8)), dim3(256), 0, stream, p);
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
  p.lens = w.lens;
  p.tile_base = w.tile_base;
  p.parts = w.parts;
  p.part_o = w.part_o;
  p.part_lse2 = w.part_lse2;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.lse2 = w.lse2;
  p.scores = w.scores;
  p.w_in = a.weights;
  p.w_out = a.weights_out;
  p.decay = a.decay;
  p.status = w.status;
  return a.head_dim == 128 ? launch_dim<128>(p, a.main_kernel_events, sms, stream)
                           : launch_dim<64>(p, a.main_kernel_events, sms, stream);
}

}  // namespace jfa
