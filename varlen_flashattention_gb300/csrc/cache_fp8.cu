// Filling and shortening the 8-bit paged KV cache (layout and scales:
// fp8_cache.cuh; the attention that reads it: decode_fp8.cu).
//
// Append: the bf16 K and V rows of new tokens, packed by offsets, become e4m3
// codes at the last positions of their sequences. For every block and head
// that receives tokens
//   need = smallest power of two >= 2^-126 with amax(new values) / need <= 448
//   s'   = need, or max(s, need) if the block already holds older tokens,
// whose codes are then re-encoded, e4m3(code * s / s'); new codes are
// e4m3(x / s'). Bound by HBM: 4 D bytes read and 2 D + 8 / block written per
// token and head.
//
// Evict: per sequence and KV head the first `first` tokens, the last `recent`
// and, up to `keep` in all, the largest weights of the rest (equal weights:
// lowest position first) move to new pages in their old order, re-encoded at
// the scale that the append's rule gives the new blocks. A selection kernel
// finds the keep-th largest weight by radix digits and lists what stays; a
// second kernel moves the rows. Bound by HBM for the move (2 (D + 4/block) + 4
// bytes read, as much written, per kept token and head) and by the latency of
// its passes for the selection.
//
// The kernels that write codes hold the values in registers between the amax and
// the encoding, so every byte is read once: a scale block by a warp, or 128
// consecutive positions of one head (whole scale blocks, a power of two up to
// 128) by a block of threads.
#include <cuda_fp16.h>

#include <algorithm>

#include "fp8_cache.cuh"

namespace jfa {

constexpr int kChunkShift = 7, kChunk = 1 << kChunkShift;  // positions of one block of threads
constexpr int kThreads = 256;

// ------------------------------------------------------------------ append

struct Fp8AppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* new_offsets;
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  int32_t batch, max_pages, page_size, total_new, max_new;
  int32_t blocks;               // scale blocks a sequence can touch, 0: found in the offsets (the kernel of short blocks)
  FastDiv by_heads, by_blocks;  // division by 2 * hkv and by `blocks`
  float* weights;
  int32_t* status;
};

__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0; }

// e4m3 codes of eight values divided by s, the quotient rounded once whatever s is:
// it is cut to fp32 with its last bit set where the division leaves a remainder, which
// fmaf gives exactly ("round to odd"), and then rounded to 4 bits. (Kept out of line,
// like recode8: the usual paths below must stay small, the kernels were losing time to
// instruction fetches with these inlined.)
__device__ __noinline__ uint2 encode8(const float* x, float s) {
  const uint32_t u = __float_as_uint(s);
  const int e = 127 - static_cast<int>(u >> 23);
  const float m = __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u);  // s = m 2^-e, 1 <= m < 2
  uint32_t r[2] = {0, 0};
#pragma unroll 1
  for (int i = 0; i < 8; i += 2) {
    float q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float y = scalbnf(x[i + k], e);  // exact but for numbers far below e4m3's smallest
      const float z = __fdiv_rz(y, m);
      const uint32_t odd = __float_as_uint(z) | (fmaf(-z, m, y) != 0.f ? 1u : 0u);
      q[k] = fabsf(x[i + k]) < INFINITY ? __uint_as_float(odd) : __int_as_float(0x7fffffff);  // infinities and NaN become NaN
    }
    r[i >> 2] |= f32x2_to_e4m3x2(q[0], q[1]) << (8 * (i & 2));
  }
  return make_uint2(r[0], r[1]);
}

// Eight codes from the scale `from` to the scale `to`, a power of two, with one
// rounding: the ratio of the scales is exact, and its product with a code, 4 by 24
// bits, is cut to 24 with its last bit set where anything was cut ("round to odd"),
// which the rounding to 4 bits cannot mistake for a tie. Out of line like encode8.
__device__ __noinline__ uint2 recode8(uint2 codes, float from, float to) {
  // Above 2^20 there are no codes but 0 (the others would pass 448); below 2^-40 nothing is left of any.
  const uint32_t u = __float_as_uint(from);
  const int e = static_cast<int>(u >> 23) - static_cast<int>(__float_as_uint(to) >> 23);
  const float ratio = __uint_as_float((static_cast<uint32_t>(min(max(e, -40), 20) + 127) << 23) | (u & 0x7FFFFFu));
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(w[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    float x[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float y = __fmul_rz(x[k], ratio);
      x[k] = __uint_as_float(__float_as_uint(y) | (fmaf(x[k], ratio, -y) != 0.f ? 1u : 0u));
    }
    r[i] = f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16);
  }
  return make_uint2(r[0], r[1]);
}

// Eight finite bf16 values divided by a power of two (inv: its inverse). The
// product is exact in bf16 but for numbers far below e4m3's smallest, so the
// codes round once.
__device__ __forceinline__ uint2 encode8_pow2(const uint4& v, __nv_bfloat162 inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), inv);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
    c[i] = f32x2_to_e4m3x2(ptx::bf16lo(u), ptx::bf16hi(u));
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

__device__ __noinline__ uint2 encode8_bf16(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = ptx::bf16lo(w[i]);
    x[2 * i + 1] = ptx::bf16hi(w[i]);
  }
  return encode8(x, s);
}

// Four codes times a power of two up to 2^15, in fp16: the product of an e4m3
// value and a power of two is exact there down to 2^-14, and what is smaller
// rounds to a zero of its sign as e4m3 either way (its smallest step is 2^-9).
__device__ __forceinline__ uint32_t scale4_pow2(uint32_t codes, __half2 ratio) {
  uint32_t lo, hi;
  e4m3x4_to_f16(codes, lo, hi);
  const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), ratio);
  const __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&hi), ratio);
  uint16_t x, y;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(x) : "r"(*reinterpret_cast<const uint32_t*>(&a)));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(*reinterpret_cast<const uint32_t*>(&b)));
  return static_cast<uint32_t>(x) | (static_cast<uint32_t>(y) << 16);
}

// The largest finite magnitude of eight bf16 values, as bf16 bits (which order
// like the magnitudes); *finite: there is nothing else among them.
__device__ __forceinline__ uint32_t amax8_bf16(const uint4& v, bool* finite) {
  const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t top = max(m & 0xFFFFu, m >> 16);
  *finite = top < 0x7F80u;
  if (!*finite) {  // infinities and NaN do not set the scale
    top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
      top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
  }
  return top;
}

// Offsets rise from 0 to total_new, and the new tokens are part of the length.
__device__ __forceinline__ bool append_range_ok(const Fp8AppendParams& p, int b, int o0, int o1, int L) {
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  return o0 >= 0 && o1 >= o0 && o1 <= p.total_new && o1 - o0 <= p.max_new && L >= o1 - o0 && L <= cap &&
         (b > 0 || o0 == 0) && (b < p.batch - 1 || o1 == p.total_new);
}

// One block checks the whole call, offsets, lengths and the pages written to, and
// sets the status block; the others pass over what is wrong without a word.
// That spares the launch that would have to clear the status block for them. A
// thread a sequence; the pages of those with many new ones are left to the warps
// (512 sequences 7 us, a warp for each 32 us). A warp reads 128 entries at a time, which the
// call waits for where pages hold one token: one prompt of 32k tokens 90 us, 43 in pages of 16
// (with blocks of one token in both).
__device__ void append_report(const Fp8AppendParams& p) {
  __shared__ int32_t s_left, s_b[kThreads], s_lo[kThreads], s_hi[kThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  auto check = [&](int b, int i) {
    const int32_t page = p.page_table[static_cast<int64_t>(b) * p.max_pages + i];
    bad |= static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.num_pages);
  };
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    if (tid == 0) s_left = 0;
    __syncthreads();
    const int b = b0 + tid;
    if (b < p.batch) {
      const int o0 = p.new_offsets[b], o1 = p.new_offsets[b + 1], L = p.seqlens[b];
      if (!append_range_ok(p, b, o0, o1, L)) {
        bad = true;
      } else if (o1 > o0) {
        const int lo = fast_div(L - (o1 - o0), p.c.page), hi = fast_div(L - 1, p.c.page);
        if (hi - lo < 4) {
          for (int i = lo; i <= hi; ++i) check(b, i);
        } else {
          const int at = atomicAdd(&s_left, 1);
          s_b[at] = b;
          s_lo[at] = lo;
          s_hi[at] = hi;
        }
      }
    }
    __syncthreads();
    for (int j = tid >> 5; j < s_left; j += kThreads / 32) {
      const int last = s_hi[j];
#pragma unroll 4
      for (int i = s_lo[j] + lane; i <= last; i += 32) check(s_b[j], i);
    }
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  if (tid < kStatusBytes / 4)
    p.status[tid] = !bad ? 0 : (tid == 0 ? JFA_ERR_BAD_INPUT : (tid == 1 ? kSiteFp8Append : 0));
}

// n consecutive positions touch at most n / c + 2 runs of c = 2^shift, so the runs of sequence b can be
// numbered from offsets[b] / c + 2 b on, all distinct. This is the sequence of such a number: the last b
// whose first one is not above it; the warp's lanes look at 32 at a time, first far apart. (Offsets that
// do not rise give some sequence.)
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int batch, int shift, int number) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0, n = batch;
  while (n > 1) {
    const uint32_t step = (n + 31) >> 5, b = lo + lane * step;
    const bool in = lane * step < n && (offsets[b] >> shift) + 2 * static_cast<int64_t>(b) <= number;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const uint32_t k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return static_cast<int>(lo);
}

// A block of threads a chunk of 128 positions of one head's K or V, for long runs in blocks too large for
// a warp's registers or too small to fill them. Bound by HBM, at 78% of the copy rate (16 prompts of
// 61 to 8192 tokens, 8 heads of 128: 77 us): the loads of a chunk are all in flight at once, four
// blocks an SM; chunks of 64, 128 or 512 threads, and K and V by the same block took 74 to 100 us.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) fp8_append_kernel(const Fp8AppendParams p) {
  constexpr int kLanes = D / 8;              // threads of a row, 8 values each
  constexpr int kRowsPerPass = kThreads / kLanes;
  constexpr int kPasses = kChunk / kRowsPerPass;
  __shared__ int32_t s_row[kChunk];          // cache row of each position, -1: nothing there to touch
  __shared__ uint32_t s_amax[kChunk];        // per scale block, bf16 bits
  __shared__ float s_new[kChunk], s_old[kChunk];
  __shared__ float s_inv[kChunk];            // 1 / s_new if that is a power of two, else 0
  constexpr int kWarpRows = 32 / kLanes;     // rows of a warp in one pass

  if (blockIdx.x == 0) {
    append_report(p);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const int hkv = p.c.hkv;
  const int unit = static_cast<int>(blockIdx.x) - 1, chunk = fast_div(unit, p.by_heads);
  const int hv = unit - chunk * 2 * hkv, h = hv >> 1;  // heads first: their rows are neighbours in memory
  const bool is_v = hv & 1;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int b = find_sequence(p.new_offsets, p.batch, kChunkShift, chunk);
  const int o0 = p.new_offsets[b], o1 = p.new_offsets[b + 1], L = p.seqlens[b];
  const int ci = chunk - (o0 / kChunk + 2 * b), f = L - (o1 - o0);  // the sequence's chunk, its first new position
  if (ci < 0 || o1 == o0 || !append_range_ok(p, b, o0, o1, L) || ci > (L - 1) / kChunk - f / kChunk) return;
  const int p0 = ((f / kChunk) + ci) * kChunk;  // this block's positions: p0 .. p0 + 127
  const int bs = p.c.block_shift;
  const int old0 = (f >> bs) << bs;            // older tokens of f's block: old0 .. f - 1
  const int sub = tid % kLanes, r0 = tid / kLanes;
  const int64_t row_elems = static_cast<int64_t>(hkv) * D;
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + (static_cast<int64_t>(o0) + p0 + r0 - f) * row_elems +
                             static_cast<int64_t>(h) * D + 8 * sub;
  uint4 raw[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    raw[k] = make_uint4(0, 0, 0, 0);
    if (static_cast<uint32_t>(p0 + r0 + k * kRowsPerPass - f) < static_cast<uint32_t>(L - f))
      raw[k] = __ldg(reinterpret_cast<const uint4*>(src + k * (kRowsPerPass * row_elems)));
  }
  if (tid < kChunk) {
    const int pos = p0 + tid;
    int row = -1;
    if (pos >= old0 && pos < L) {
      const int pg = fast_div(pos, p.c.page);
      const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pg];
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.c.num_pages))
        row = page * p.page_size + (pos - pg * p.page_size);
    }
    s_row[tid] = row;
    s_amax[tid] = 0;
    if (p.weights && !is_v && pos >= f && pos < L)
      p.weights[(static_cast<int64_t>(b) * hkv + h) * cap + pos] = 0.f;
  }
  __syncthreads();
  uint32_t odd = 0;  // rows of this thread that hold infinities or NaN
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    bool finite;
    uint32_t a = amax8_bf16(raw[k], &finite);
    if (!finite) odd |= 1u << k;
    if ((1 << bs) >= kWarpRows) {  // the warp's rows are of one block
      a = __reduce_max_sync(0xffffffffu, a);
      if (lane == 0) atomicMax(&s_amax[(k * kRowsPerPass + r0) >> bs], a);
    } else {
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
      if (sub == 0) atomicMax(&s_amax[(k * kRowsPerPass + r0) >> bs], a);
    }
  }
  __syncthreads();
  float* scales = is_v ? p.c.vs : p.c.ks;
  if (tid < (kChunk >> bs)) {
    const int start = p0 + (tid << bs);
    const int pos = max(start, f);  // the block's first new position, if it has one
    if (pos < min(L, start + (1 << bs)) && s_row[pos - p0] >= 0) {
      float s = e4m3_block_scale(__uint_as_float(s_amax[tid] << 16));
      float* cell = scales + static_cast<int64_t>(s_row[pos - p0] >> bs) * hkv + h;
      const float old = start < f ? *cell : 0.f;
      s = fmaxf(s, old);
      s_old[tid] = start < f ? old : s;
      s_new[tid] = s;
      s_inv[tid] = is_pow2(s) ? 1.f / s : 0.f;
      *cell = s;
    }
  }
  __syncthreads();
  uint8_t* codes = (is_v ? p.c.vc : p.c.kc) + static_cast<int64_t>(h) * D + 8 * sub;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int t = k * kRowsPerPass + r0, pos = p0 + t;
    const int row = s_row[t];
    if (row < 0) continue;
    uint2* dst = reinterpret_cast<uint2*>(codes + row * row_elems);
    const float inv = s_inv[t >> bs];
    if (pos >= f) {
      *dst = inv != 0.f && !((odd >> k) & 1) ? encode8_pow2(raw[k], __float2bfloat162_rn(inv))
                                              : encode8_bf16(raw[k], s_new[t >> bs]);
    } else if (s_old[t >> bs] != s_new[t >> bs]) {  // an older token of a block whose scale has grown
      *dst = recode8(*dst, s_old[t >> bs], s_new[t >> bs]);
    }
  }
}

// A warp a scale block: its new rows, ROWS at most, stay in the warp's registers, and nothing but the
// warp's own reduction lies between their loads and the stores, where the chunks' blocks of threads wait
// at three barriers. Bound by HBM for prompts, by the chain of loads (offsets and length, page, old
// scale) for a step's tokens.
template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS > 16 ? 2 : 4) fp8_append_warp_kernel(const Fp8AppendParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, 8 values each; rows of a warp
  if (blockIdx.x == 0) {
    append_report(p);
    return;
  }
  const int lane = threadIdx.x & 31, sub = lane % kLanes, r0 = lane / kLanes;
  const int hkv = p.c.hkv, bs = p.c.block_shift;
  const int job = (static_cast<int>(blockIdx.x) - 1) * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const int unit = fast_div(job, p.by_heads), hv = job - unit * 2 * hkv, h = hv >> 1;
  const bool is_v = hv & 1;
  const int b = p.blocks ? fast_div(unit, p.by_blocks) : find_sequence(p.new_offsets, p.batch, bs, unit);
  if (b >= p.batch) return;
  const int o0 = p.new_offsets[b], o1 = p.new_offsets[b + 1], L = p.seqlens[b];
  const int f = L - (o1 - o0);  // the first new position
  const int bi = unit - (p.blocks ? b * p.blocks : (o0 >> bs) + 2 * b);  // the sequence's block
  if (o1 == o0 || bi < 0 || !append_range_ok(p, b, o0, o1, L) || bi > ((L - 1) >> bs) - (f >> bs)) return;
  const int start = ((f >> bs) + bi) << bs;  // the block's first position
  const int pg = fast_div(start, p.c.page);
  const int64_t row_elems = static_cast<int64_t>(hkv) * D;
  const int lo = max(start, f), hi = min(L, start + (1 << bs));  // its new positions
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + (static_cast<int64_t>(o0) + lo - f) * row_elems +
                             static_cast<int64_t>(h) * D + 8 * sub;
  constexpr int kMost = ROWS / kRows;  // passes over the new rows
  uint4 raw[kMost];
  uint32_t top = 0, odd = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int i = k * kRows + r0;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (lo + i < hi) raw[k] = __ldg(reinterpret_cast<const uint4*>(src + i * row_elems));
  }
  const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pg];
  if (p.weights && !is_v && lane < hi - lo)
    p.weights[(static_cast<int64_t>(b) * hkv + h) * (static_cast<int64_t>(p.max_pages) * p.page_size) + lo + lane] = 0.f;
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.num_pages)) return;
  const int row = page * p.page_size + (start - pg * p.page_size);  // of the block's first position
  float* cell = (is_v ? p.c.vs : p.c.ks) + static_cast<int64_t>(row >> bs) * hkv + h;
  const float old = start < f ? *cell : 0.f;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    bool finite;
    top = max(top, amax8_bf16(raw[k], &finite));
    if (!finite) odd |= 1u << k;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const float s = fmaxf(e4m3_block_scale(__uint_as_float(top << 16)), old);
  __syncwarp();  // every lane has read the cell
  if (lane == 0) *cell = s;
  const float inv = is_pow2(s) ? 1.f / s : 0.f;
  uint8_t* codes = (is_v ? p.c.vc : p.c.kc) + row * row_elems + static_cast<int64_t>(h) * D + 8 * sub;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int pos = lo + k * kRows + r0;
    if (pos < hi)
      *reinterpret_cast<uint2*>(codes + (pos - start) * row_elems) =
          inv != 0.f && !((odd >> k) & 1) ? encode8_pow2(raw[k], __float2bfloat162_rn(inv)) : encode8_bf16(raw[k], s);
  }
  if (start < f && s != old) {  // the older tokens of a block whose scale has grown
    for (int pos = start + r0; pos < f; pos += kRows) {
      uint2* dst = reinterpret_cast<uint2*>(codes + (pos - start) * row_elems);
      *dst = recode8(*dst, old, s);
    }
  }
}

cudaError_t launch_cache_append_fp8(const jfa_cache_append_fp8_args& a, int32_t* status, cudaStream_t stream) {
  Fp8AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.new_offsets = a.new_offsets;
  p.c.kc = static_cast<uint8_t*>(a.k_cache);
  p.c.vc = static_cast<uint8_t*>(a.v_cache);
  p.c.ks = a.k_scale;
  p.c.vs = a.v_scale;
  p.c.hkv = a.kv_heads;
  p.c.num_pages = a.num_pages;
  p.c.block_shift = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.c.page = make_fast_div(a.page_size);
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.batch = a.batch;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.total_new = a.total_new;
  p.max_new = a.max_new;
  p.by_heads = make_fast_div(2 * a.kv_heads);
  p.weights = a.weights;
  p.status = status;
  const int64_t heads = 2 * static_cast<int64_t>(a.kv_heads);
  // A warp a scale block where the block's rows fit its registers and are not few among many: of 8 heads
  // of 128, 16 prompts of 61 to 8192 tokens take 67 us with blocks of 16 tokens (77 by chunks), 75 with
  // blocks of 32 (77), but 100 with blocks of 8 (77), a row or so a warp. The same of one head 9.8 (12.0),
  // 11.6 (12.0) and 14.1 (12.0), and of head_dim 64, where a warp covers four rows a pass instead of two: 8 heads
  // 44 (49), 49 (50) and 69 (49), one head 7.1 (7.5), 7.5 (7.7) and 10.1 (7.9). Of few new tokens it is the
  // faster one whatever the block: 512 x 1 token 6.9 us (66), 256 x 32 in blocks of 128 12.4 (35; of head_dim
  // 64 8.7 and 26; of one head 5.4 and 7.6), 256 x 16 in blocks of 1 37 (35 to 40; one head 7.0 and 7.4).
  const int64_t fixed = (static_cast<int64_t>(a.max_new) + a.block_size - 2) / a.block_size + 1;
  const int64_t most = a.total_new / a.block_size + 2 * static_cast<int64_t>(a.batch);
  const int64_t jobs = std::min(fixed * a.batch, most) * heads;
  const bool short_blocks = a.max_new <= 16 || (a.block_size >= 16 && std::min(a.max_new, a.block_size) <= 32);
  if (short_blocks && jobs < (int64_t(1) << 31) - 64) {
    p.blocks = fixed * a.batch <= most ? static_cast<int32_t>(fixed) : 0;
    p.by_blocks = make_fast_div(std::max(p.blocks, 1));
    const uint32_t grid = static_cast<uint32_t>((jobs + kThreads / 32 - 1) / (kThreads / 32)) + 1;
    if (std::min(a.max_new, a.block_size) <= 16) {
      if (a.head_dim == 128)
        fp8_append_warp_kernel<128, 16><<<grid, kThreads, 0, stream>>>(p);
      else
        fp8_append_warp_kernel<64, 16><<<grid, kThreads, 0, stream>>>(p);
    } else {
      if (a.head_dim == 128)
        fp8_append_warp_kernel<128, 32><<<grid, kThreads, 0, stream>>>(p);
      else
        fp8_append_warp_kernel<64, 32><<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
  }
  const uint32_t grid = static_cast<uint32_t>((a.total_new / kChunk + 2 * static_cast<int64_t>(a.batch)) * heads) + 1;
  if (a.head_dim == 128)
    fp8_append_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else
    fp8_append_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ evict

struct Fp8EvictParams {
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* new_table;
  const float* weights;
  int32_t batch, max_pages, new_max_pages, page_size, keep, first, recent, chunks;
  FastDiv by_heads, by_chunks;  // division by hkv and by chunks
  int32_t* kept;         // [B, hkv, keep]
  int32_t* new_seqlens;  // [B]
  float* new_weights;    // [B, hkv, new_max_pages * page_size]
  uint8_t* page_ok;      // [B, new_max_pages]: the new page may be written
  int32_t bitmap_words;  // of the pages' bitmaps in shared memory
  int32_t shrink;        // short sequences leave blocks of their clusters to others
  int32_t* status;
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMostBitmapWords = 8192;  // two bitmaps of 32 KB (two blocks still fit an SM): runs of 262,144 pages

// Order of the weights as unsigned numbers; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w == w ? w + 0.f : -INFINITY);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// What stays of one sequence and KV head, in order: a cluster of blocks, each
// with a run of the candidates, each warp with a run of the block's. A thread
// reads its keys once, 32 apart, and keeps KEYS of them in registers (longer
// runs, past 8 x 16,384 candidates, are read again for every pass). The
// threshold is found by up to four digits of 8 bits (fewer where all keys with the
// digits so far stay: 32 sequences of 1k-32k 88 -> 84 us), counted in shared memory (equal
// digits of a warp cost no more than different ones) and added into every block
// of the cluster through distributed shared memory (stores and additions there
// overlap, loads of the 8 blocks' counts took 1.7 us a pass), where one warp of
// each finds the same digit; then the blocks list their survivors, placed by the numbers
// of survivors before them. This is bound by instructions and by the latency of
// its few dependent steps, not by bytes: hence few warps with many keys, a key
// of 0, below every weight's, where a thread has none, instead of tests, small
// digits (11 bits take a pass less, but 2048 counts from each of 8 blocks took
// 2.8 us a pass), places from byte sums of four steps at once (population counts
// run at an eighth of the rate), and no store to global memory before the
// cluster's last barrier, which would wait for it.
struct alignas(16) SelShared {
  int32_t hist[4][256];      // this block's counts
  int32_t sum[4][256];       // the cluster's
  int32_t warp_sum[2][32];
  int32_t count[2][8];       // survivors above the threshold (or all), and equal to it, of each block
  uint32_t digit;
  int32_t left;              // how many keys with the prefix found so far stay
  int32_t hits;              // how many there are
};

// Every sequence's first `used(b)` entries of a table, each once, by one block: all threads on one
// sequence after the other, or a warp a sequence, the lengths of 32 at once and the next one's first
// entries on their way (512 sequences of up to 2k tokens 267 us the call, 294 one after the other);
// whichever takes fewer steps where the rows are full (15 x 20k-32k tokens in pages of 16: a warp each
// 29 us, all on each 40). f(b, i, entry) is called by the thread that read the entry. One block is enough
// for pages of 16 tokens; with pages of one token the call waits for it (32 x 1k-32k tokens cut to 2k
// 701 us, 89 in pages of 16 with blocks of one token; one of 131k cut to 16k 96 and 29).
template <class Used, class F>
__device__ __forceinline__ void for_entries(const int32_t* table, int batch, int width, Used used, F f) {
  const int lane = threadIdx.x & 31;
  auto fetch = [&](int b, int n, int i0, int stride, int32_t (&v)[8]) {
    const int32_t* row = table + static_cast<int64_t>(b) * width;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i0 + k * stride < n ? row[i0 + k * stride] : 0;
  };
  auto visit = [&](int b, int n, int i0, int stride, const int32_t (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * stride < n) f(b, i0 + k * stride, v[k]);
  };
  const int64_t steps_all = batch * static_cast<int64_t>(width / (8 * kSelThreads) + 1);
  if (steps_all <= ((batch - 1) / kSelWarps + 1) * static_cast<int64_t>(width / 256 + 1)) {
    for (int b = 0; b < batch; ++b) {
      const int n = used(b);
      for (int i0 = threadIdx.x; i0 < n; i0 += 8 * kSelThreads) {
        int32_t v[8];
        fetch(b, n, i0, kSelThreads, v);
        visit(b, n, i0, kSelThreads, v);
      }
    }
    return;
  }
  for (int b0 = threadIdx.x >> 5; b0 < batch; b0 += 32 * kSelWarps) {
    const int mine = b0 + lane * kSelWarps, many = min(32, (batch - b0 + kSelWarps - 1) / kSelWarps);
    const int n_mine = mine < batch ? used(mine) : 0;
    int n = __shfl_sync(0xffffffffu, n_mine, 0);
    int32_t v[8], next[8];
    fetch(b0, n, lane, 32, v);
    for (int j = 0; j < many; ++j) {
      const int b = b0 + j * kSelWarps, n_next = j + 1 < many ? __shfl_sync(0xffffffffu, n_mine, j + 1) : 0;
      fetch(b + kSelWarps, n_next, lane, 32, next);
      visit(b, n, lane, 32, v);
      for (int i0 = lane + 256; i0 < n; i0 += 256) {
        fetch(b, n, i0, 32, v);
        visit(b, n, i0, 32, v);
      }
      n = n_next;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = next[k];
    }
  }
}

// One block checks the call beside the selection: lengths, table entries, and
// that no new page is one that a sequence still reads or is given out twice.
// It sets the status block and, for each new page in use, whether the move may
// write to it; the other blocks pass over what is wrong without a word. That
// spares the launch that would have to clear the status block, and counters of
// pages in memory, for them.
__device__ void evict_check(const Fp8EvictParams& p, uint32_t* bitmap) {
  uint32_t *taken = bitmap, *bad_page = bitmap + p.bitmap_words;  // read from or given out; given out wrongly
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  bool bad = false;
  auto length = [&](int b) {
    const int L = p.seqlens[b];
    const bool wrong = L < 0 || L > cap || (L > 0 && p.c.num_pages == 0);
    bad |= wrong;
    return wrong ? 0 : L;
  };
  auto used = [&](int b) {
    const int L = length(b);
    return L > 0 ? fast_div(L - 1, p.c.page) + 1 : 0;
  };
  auto fresh = [&](int b) {
    const int n = min(length(b), p.keep);
    return n > 0 ? fast_div(n - 1, p.c.page) + 1 : 0;
  };
  const uint32_t pages = static_cast<uint32_t>(p.c.num_pages), run = static_cast<uint32_t>(p.bitmap_words) * 32u;
  for (uint32_t base = 0; base == 0 || base < pages; base += run) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.bitmap_words; i += kSelThreads) bitmap[i] = 0;
    __syncthreads();
    for_entries(p.page_table, p.batch, p.max_pages, used, [&](int, int, int32_t page) {
      const uint32_t i = static_cast<uint32_t>(page) - base;
      bad |= static_cast<uint32_t>(page) >= pages;
      if (static_cast<uint32_t>(page) < pages && i < run) atomicOr(&taken[i >> 5], 1u << (i & 31));
    });
    __syncthreads();
    for_entries(p.new_table, p.batch, p.new_max_pages, fresh, [&](int, int, int32_t page) {
      const uint32_t i = static_cast<uint32_t>(page) - base, bit = 1u << (i & 31);
      if (static_cast<uint32_t>(page) < pages && i < run && (atomicOr(&taken[i >> 5], bit) & bit))
        atomicOr(&bad_page[i >> 5], bit);
    });
    __syncthreads();
    for_entries(p.new_table, p.batch, p.new_max_pages, fresh, [&](int b, int j, int32_t page) {
      const uint32_t i = static_cast<uint32_t>(page) - base;
      const bool in = static_cast<uint32_t>(page) < pages;
      if (in ? i >= run : base > 0) return;  // another run's
      const bool ok = in && !((bad_page[i >> 5] >> (i & 31)) & 1);
      p.page_ok[static_cast<int64_t>(b) * p.new_max_pages + j] = ok;
      bad |= !ok;
    });
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x < kStatusBytes / 4)
    p.status[threadIdx.x] = !bad ? 0 : (threadIdx.x == 0 ? JFA_ERR_BAD_INPUT : (threadIdx.x == 1 ? kSiteFp8Evict : 0));
}

template <int KEYS>
__global__ void __launch_bounds__(kSelThreads, KEYS <= 16 ? 2 : 1)
    fp8_evict_select_kernel(const Fp8EvictParams p, int cluster) {
  __shared__ SelShared sh;
  extern __shared__ uint32_t s_bitmap[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int>(blockIdx.x) < cluster) {
    allow_next_grid();
    if (blockIdx.x == 0) evict_check(p, s_bitmap);
    return;
  }
  const int seg = static_cast<int>(blockIdx.x) / cluster - 1;  // the first cluster's first block checks the call
  const int b = seg / p.c.hkv, h = seg % p.c.hkv;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int new_cap = p.new_max_pages * p.page_size;
  int L = p.seqlens[b];
  if (L < 0 || L > cap || (L > 0 && p.c.num_pages == 0)) L = 0;
  const bool choose = L > p.keep && p.keep > p.first + p.recent;
  // The cluster is made for a full row of the table. Where not all clusters are on the device at
  // once, a shorter sequence takes as many of the blocks as its keys (or the zeros behind what is
  // kept) fill, and the others leave: 32 x 1k-8k tokens in rows of 131k 59 us, 137 us
  // without. (Barriers of a cluster wait for the threads that have not left.)
  const int rank = cluster > 1 ? static_cast<int>(blockIdx.x % cluster) : 0;
  if (cluster > 1 && p.shrink) {
    const int work = max(choose ? L - p.recent - p.first : 0, new_cap), each = KEYS * kSelThreads;
    cluster = min(cluster, max(1, (work - 1) / each + 1));
    if (rank >= cluster) return;
  }
  reinterpret_cast<int4*>(sh.hist)[tid] = make_int4(0, 0, 0, 0);  // 512 threads: hist and sum
  static_assert(kSelThreads * 16 == sizeof(sh.hist) + sizeof(sh.sum), "one int4 a thread clears both");
  if (cluster > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // waited for before the first addition
  allow_next_grid();
  const int wide = cluster * kSelThreads, wtid = rank * kSelThreads + tid;  // threads of the cluster
  const int n = min(L, p.keep);
  const float* w = p.weights + seg * cap;
  int32_t* kept = p.kept + static_cast<int64_t>(seg) * p.keep;
  float* nw = p.new_weights + static_cast<int64_t>(seg) * new_cap;

  // the candidates c0 .. c1 - 1, and this warp's run lo .. hi - 1 of them
  const int c0 = p.first, c1 = max(L - p.recent, c0);
  const int runs = cluster * kSelWarps;
  const int per_warp = choose ? ((c1 - c0 + runs - 1) / runs + 31) / 32 * 32 : 0;
  const int lo = static_cast<int>(min(c0 + static_cast<int64_t>(rank * kSelWarps + warp) * per_warp, static_cast<int64_t>(c1)));
  const int count = choose ? min(lo + per_warp, c1) - lo - lane : 0;  // keys at w[lo + lane + 32 c], 32 c < count
  w += lo + lane;
  const int steps = per_warp / 32;
  uint32_t key[KEYS];
  {
    float x[KEYS];
#pragma unroll
    for (int c = 0; c < KEYS; ++c) {
      x[c] = 0.f;
      if (32 * c < count) x[c] = __ldg(w + 32 * c);
    }
    __syncthreads();  // the counts are zero
#pragma unroll
    for (int c = 0; c < KEYS; ++c) {
      key[c] = 0u;
    }
#pragma unroll
    for (int g = 0; g < KEYS; g += 4) {
      if (g >= steps) break;
#pragma unroll
      for (int c = g; c < g + 4; ++c) {
        if (32 * c < count) key[c] = weight_key(x[c]);
        atomicAdd(&sh.hist[0][key[c] >> 24], 1);
      }
    }
  }
  auto late_key = [&](int c) -> uint32_t { return 32 * c < count ? weight_key(__ldg(w + 32 * c)) : 0u; };
#pragma unroll 1
  for (int c = KEYS; c < steps; ++c) atomicAdd(&sh.hist[0][late_key(c) >> 24], 1);
  // Everything but the candidates' places: what is certain to stay, and zeros.
  auto finish = [&] {
    if (h == 0 && wtid == 0) p.new_seqlens[b] = n;
    for (int j = n + wtid; j < p.keep; j += wide) kept[j] = -1;
    for (int j = n + wtid; j < new_cap; j += wide) nw[j] = 0.f;
    if (L <= p.keep) {
      for (int j = wtid; j < n; j += wide) kept[j] = j;
    } else {
      for (int j = wtid; j < p.first; j += wide) kept[j] = j;
      for (int j = wtid; j < p.recent; j += wide) kept[p.keep - p.recent + j] = c1 + j;
    }
  };
  if (!choose) {  // the same in all blocks of the cluster
    if (cluster > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    finish();
    return;
  }

  auto cluster_sync = [&] {
    if (cluster > 1) {
      asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  auto remote = [&](const int32_t* local, int r) -> uint32_t {  // the address of block r's copy
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(local)), "r"(r));
    return at;
  };

  // The need-th largest key, digit by digit from the top.
  uint32_t prefix = 0;
  int need = p.keep - p.first - p.recent;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    if (pass > 0) {
      const int above = 32 - 8 * pass, shift = 24 - 8 * pass;
#pragma unroll
      for (int g = 0; g < KEYS; g += 4) {
        if (g >= steps) break;
#pragma unroll
        for (int c = g; c < g + 4; ++c)
          if ((key[c] >> above) == prefix) atomicAdd(&sh.hist[pass][(key[c] >> shift) & 255], 1);
      }
#pragma unroll 1
      for (int c = KEYS; c < steps; ++c) {
        const uint32_t k = late_key(c);
        if ((k >> above) == prefix) atomicAdd(&sh.hist[pass][(k >> shift) & 255], 1);
      }
    }
    const int32_t* bins = sh.hist[pass];
    __syncthreads();
    if (cluster > 1) {
      if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (tid < 256) {
        const int32_t v = sh.hist[pass][tid];
        if (v)
          for (int r = 0; r < cluster; ++r)
            asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(remote(&sh.sum[pass][tid], r)),
                         "r"(v)
                         : "memory");
      }
      cluster_sync();
      bins = sh.sum[pass];
    }
    if (warp == 0) {
      // lane l holds the digits 255 - 8 l down to 248 - 8 l
      const int4 d = *reinterpret_cast<const int4*>(bins + 248 - 8 * lane);
      const int4 u = *reinterpret_cast<const int4*>(bins + 252 - 8 * lane);
      const int cnt[8] = {u.w, u.z, u.y, u.x, d.w, d.z, d.y, d.x};
      int own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += cnt[i];
      int upto = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      int before = upto - own;
      if (before < need && upto >= need) {  // one lane: the digit is one of its own
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + cnt[i] >= need) {
            sh.digit = 255 - 8 * lane - i;
            sh.left = need - before;
            sh.hits = cnt[i];
          }
          before += cnt[i];
        }
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | sh.digit;
    need = sh.left;
    // Every key with these digits stays: the digits below do not matter. (Then no key of
    // 0 is among them, the keys that stay are weights.)
    if (sh.hits == need) {
      prefix <<= 24 - 8 * pass;
      break;
    }
  }
  // Keys above `prefix` stay, and the first `need` of the sh.hits that equal it.
  // Where all of those do, which is the usual case, no rank among them is needed.
  const bool all_equal = sh.hits == need;
  int gt = 0, eq = 0;
  if (all_equal) {
#pragma unroll
    for (int g = 0; g < KEYS; g += 4) {
      if (g >= steps) break;
#pragma unroll
      for (int c = g; c < g + 4; ++c) gt += key[c] >= prefix;
    }
  } else {
#pragma unroll
    for (int c = 0; c < KEYS; ++c) {
      gt += key[c] > prefix;
      eq += key[c] == prefix;
    }
  }
#pragma unroll 1
  for (int c = KEYS; c < steps; ++c) {
    const uint32_t k = late_key(c);
    gt += k > prefix || (all_equal && k == prefix);
    eq += !all_equal && k == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  // before this warp: the block's earlier warps, the cluster's earlier blocks
  if (lane == 0) {
    sh.warp_sum[0][warp] = gt;
    sh.warp_sum[1][warp] = eq;
  }
  __syncthreads();
  const int vg = lane < kSelWarps ? sh.warp_sum[0][lane] : 0, ve = lane < kSelWarps ? sh.warp_sum[1][lane] : 0;
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? vg : 0);
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? ve : 0);
  if (cluster > 1) {
    if (warp == 0) {
      const int all_gt = __reduce_add_sync(0xffffffffu, vg), all_eq = __reduce_add_sync(0xffffffffu, ve);
      if (lane < cluster) {
        asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.count[0][rank], lane)), "r"(all_gt) : "memory");
        asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(remote(&sh.count[1][rank], lane)), "r"(all_eq) : "memory");
      }
    }
    cluster_sync();  // and the last: nothing reaches into another block after it
    gt0 += __reduce_add_sync(0xffffffffu, lane < rank ? sh.count[0][lane] : 0);
    eq0 += __reduce_add_sync(0xffffffffu, lane < rank ? sh.count[1][lane] : 0);
  }
  int32_t* out = kept + p.first;
  const int t0 = lo + lane;
  if (all_equal) {
#pragma unroll
    for (int c = 0; c < KEYS; c += 4) {
      if (c >= steps) break;
      // byte i: the survivors of step c + i up to this lane
      uint32_t own = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) own |= (key[c + i] >= prefix ? 1u : 0u) << (8 * i);
      uint32_t upto = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      const uint32_t whole = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (key[c + i] >= prefix) out[gt0 + static_cast<int>((upto >> (8 * i)) & 255) - 1] = t0 + 32 * (c + i);
        gt0 += static_cast<int>((whole >> (8 * i)) & 255);
      }
    }
  }
  const uint32_t below = (1u << lane) - 1;
  auto place = [&](int c, uint32_t k) {  // one step, with ranks among equal keys
    const uint32_t mg = __ballot_sync(0xffffffffu, k > prefix);
    const uint32_t me = __ballot_sync(0xffffffffu, k == prefix);
    const int eq_rank = eq0 + __popc(me & below);
    const int j = gt0 + __popc(mg & below) + min(eq_rank, need);
    if (k > prefix || (k == prefix && eq_rank < need)) out[j] = t0 + 32 * c;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  };
  auto place_all = [&](int c, uint32_t k) {  // one step, every equal key stays
    const uint32_t m = __ballot_sync(0xffffffffu, k >= prefix);
    if (k >= prefix) out[gt0 + __popc(m & below)] = t0 + 32 * c;
    gt0 += __popc(m);
  };
  if (!all_equal) {
#pragma unroll
    for (int c = 0; c < KEYS; ++c)
      if (c < steps) place(c, key[c]);
  }
#pragma unroll 1
  for (int c = KEYS; c < steps; ++c) {
    if (all_equal)
      place_all(c, late_key(c));
    else
      place(c, late_key(c));
  }
  finish();
}

// Moves the kept rows, 128 new positions of one head, K and V, at a time. What
// finds a row is a chain of loads (kept position, page, state of the new page)
// longer than the row's own, so the blocks stay and look up the next chunk's
// rows while this one's are on their way.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) fp8_evict_move_kernel(const Fp8EvictParams p, int jobs) {
  constexpr int kLanes = D / 16;             // threads of a row, 16 codes each
  constexpr int kRowsPerPass = kThreads / kLanes;
  constexpr int kPasses = kChunk / kRowsPerPass;
  __shared__ int32_t s_src[2][kChunk], s_dst[2][kChunk];  // cache rows, -1: none
  __shared__ uint32_t s_amax[2][kChunk];
  __shared__ float s_new[2][kChunk];

  const int hkv = p.c.hkv, bs = p.c.block_shift, tid = threadIdx.x;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t new_cap = static_cast<int64_t>(p.new_max_pages) * p.page_size;
  const int sub = tid % kLanes, r0 = tid / kLanes;
  const int blocks = kChunk >> bs;
  // job = (sequence, chunk, head), heads first
  auto place = [&](int job, int& b, int& j0, int& h) {
    const int chunk = fast_div(job, p.by_heads);
    h = job - chunk * hkv;
    b = fast_div(chunk, p.by_chunks);
    j0 = (chunk - b * p.chunks) * kChunk;
  };
  // This block's jobs that have rows, 32 looked at together, so that those of empty or short sequences
  // cost next to nothing (512 sequences of which 8 hold 16k-32k tokens: 114 us the call, 446 us without).
  const int step = gridDim.x;
  int64_t scan = static_cast<int64_t>(blockIdx.x) - 32 * step;
  uint32_t found = 0;  // among scan, scan + step, ...
  auto next_job = [&]() -> int {
    while (!found) {
      scan += 32 * step;
      if (scan >= jobs) return jobs;
      const int64_t job = scan + (tid & 31) * step;
      bool rows = false;
      if (job < jobs) {
        int b, j0, h;
        place(static_cast<int>(job), b, j0, h);
        const int L = p.seqlens[b];
        rows = L > j0 && L <= cap;
      }
      found = __ballot_sync(0xffffffffu, rows);
    }
    const int i = __ffs(found) - 1;
    found &= found - 1;
    return static_cast<int>(scan) + i * step;
  };
  auto kept_of = [&](int job) -> int {  // old position of this thread's new one, -1: none
    if (job >= jobs || tid >= kChunk) return -1;
    int b, j0, h;
    place(job, b, j0, h);
    return j0 + tid < p.keep ? p.kept[(static_cast<int64_t>(b) * hkv + h) * p.keep + j0 + tid] : -1;
  };
  auto look_up = [&](int job, int t, int buf) {
    if (job >= jobs || tid >= kChunk) return;
    int src = -1, dst = -1;
    if (t >= 0) {
      int b, j0, h;
      place(job, b, j0, h);
      const int j = j0 + tid;
      const int64_t seg = static_cast<int64_t>(b) * hkv + h;
      const float weight = p.weights[seg * cap + t];
      const int pg = fast_div(t, p.c.page), npg = fast_div(j, p.c.page);
      const uint32_t page = static_cast<uint32_t>(p.page_table[static_cast<int64_t>(b) * p.max_pages + pg]);
      const uint32_t fresh = static_cast<uint32_t>(p.new_table[static_cast<int64_t>(b) * p.new_max_pages + npg]);
      const uint32_t pages = static_cast<uint32_t>(p.c.num_pages);
      if (page < pages) src = static_cast<int>(page) * p.page_size + (t - pg * p.page_size);
      if (p.page_ok[static_cast<int64_t>(b) * p.new_max_pages + npg])  // then it is one of the pages
        dst = static_cast<int>(fresh) * p.page_size + (j - npg * p.page_size);
      p.new_weights[seg * new_cap + j] = weight;
    }
    s_src[buf][tid] = src;
    s_dst[buf][tid] = dst;
  };
  int job = next_job(), next = next_job();
  wait_prior_grid();
  int t_next = kept_of(job);
  look_up(job, t_next, 0);
  t_next = kept_of(next);
  for (int buf = 0; job < jobs; buf ^= 1) {
    if (tid < kChunk) s_amax[0][tid] = s_amax[1][tid] = 0;
    __syncthreads();  // this chunk's rows are known
    int b, j0, h;
    place(job, b, j0, h);
    uint8_t* codes[2] = {p.c.kc + static_cast<int64_t>(h) * D + 16 * sub, p.c.vc + static_cast<int64_t>(h) * D + 16 * sub};
    float* scales[2] = {p.c.ks + h, p.c.vs + h};
    uint4 raw[2][kPasses];
    float sc[2][kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int src = s_src[buf][k * kRowsPerPass + r0];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        raw[v][k] = make_uint4(0, 0, 0, 0);  // a token whose page is missing becomes zeros
        sc[v][k] = 0.f;
        if (src >= 0) {
          raw[v][k] = *reinterpret_cast<const uint4*>(codes[v] + static_cast<int64_t>(src) * hkv * D);
          sc[v][k] = scales[v][static_cast<int64_t>(src >> bs) * hkv];
        }
      }
    }
    look_up(next, t_next, buf ^ 1);
    job = next;
    next = next_job();
    t_next = kept_of(next);
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t w[4] = {raw[v][k].x, raw[v][k].y, raw[v][k].z, raw[v][k].w};
        __half2 top = __float2half2_rn(0.f);  // largest magnitude; the maximum passes over NaN
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo, hi;
          e4m3x4_to_f16(w[i] & 0x7F7F7F7Fu, lo, hi);
          top = __hmax2(top, __hmax2(*reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&hi)));
        }
        float a = __half2float(__hmax(__low2half(top), __high2half(top)));
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        // in units of 2^8, which keeps values past fp32's range (a scale of 2^127 holds 448 * 2^127), rounded up:
        // never past 1.75 times a power of two, the border of e4m3_block_scale_from_256th
        if (sub == 0) atomicMax(&s_amax[v][(k * kRowsPerPass + r0) >> bs], __float_as_uint(__fmul_ru(a * 0x1p-8f, sc[v][k])));
      }
    }
    __syncthreads();
    if (tid < 2 * blocks) {
      const int v = tid >= blocks, i = tid - v * blocks;
      const float s = e4m3_block_scale_from_256th(__uint_as_float(s_amax[v][i]));
      s_new[v][i] = s;
      const int dst = s_dst[buf][i << bs];
      if (dst >= 0) scales[v][static_cast<int64_t>(dst >> bs) * hkv] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int t = k * kRowsPerPass + r0;
      const int dst = s_dst[buf][t];
      if (dst < 0) continue;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float s = s_new[v][t >> bs], from = sc[v][k];
        uint4 out = raw[v][k];
        if (s != from) {
          // both powers of two: the ratio is one, and is exact; below fp16's range nothing is left of the codes
          const float ratio = from / s;
          if (is_pow2(from) && ratio <= 32768.f) {
            const __half2 r = __float2half2_rn(ratio);
            out = make_uint4(scale4_pow2(out.x, r), scale4_pow2(out.y, r), scale4_pow2(out.z, r), scale4_pow2(out.w, r));
          } else {
            const uint2 lo = recode8(make_uint2(out.x, out.y), from, s), hi = recode8(make_uint2(out.z, out.w), from, s);
            out = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
        }
        *reinterpret_cast<uint4*>(codes[v] + static_cast<int64_t>(dst) * hkv * D) = out;
      }
    }
  }
}

template <int KEYS>
static cudaError_t launch_select_keys(Fp8EvictParams& p, int cluster, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((static_cast<uint32_t>(p.batch) * p.c.hkv + 1) * cluster);
  p.shrink = cfg.gridDim.x > static_cast<uint32_t>(sms) * (KEYS <= 16 ? 2 : 1);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.bitmap_words) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(fp8_evict_select_kernel<KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMostBitmapWords * 8);
  });
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, fp8_evict_select_kernel<KEYS>, p, cluster);
}

// By the candidates that a full row of the page table can hold: one block for up to 8192 (4 keys a
// thread up to 2048, else 16), clusters of up to 8 blocks (the portable size) past that, and
// 32 keys a thread past 65,536.
static cudaError_t launch_select(Fp8EvictParams& p, int sms, cudaStream_t stream) {
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  if (cap <= 4 * kSelThreads) return launch_select_keys<4>(p, 1, sms, stream);
  int cluster = 1;
  while (cluster < 8 && cap > static_cast<int64_t>(cluster) * 16 * kSelThreads) cluster *= 2;
  return cap <= static_cast<int64_t>(cluster) * 16 * kSelThreads ? launch_select_keys<16>(p, cluster, sms, stream)
                                                                 : launch_select_keys<32>(p, cluster, sms, stream);
}

cudaError_t launch_cache_evict_fp8(const jfa_cache_evict_fp8_args& a, uint8_t* page_ok, int32_t* status, int sms,
                                   cudaStream_t stream) {
  Fp8EvictParams p{};
  p.c.kc = static_cast<uint8_t*>(a.k_cache);
  p.c.vc = static_cast<uint8_t*>(a.v_cache);
  p.c.ks = a.k_scale;
  p.c.vs = a.v_scale;
  p.c.hkv = a.kv_heads;
  p.c.num_pages = a.num_pages;
  p.c.block_shift = __builtin_ctz(static_cast<unsigned>(a.block_size));
  p.c.page = make_fast_div(a.page_size);
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.new_table = a.new_page_table;
  p.weights = a.weights;
  p.batch = a.batch;
  p.max_pages = a.max_pages;
  p.new_max_pages = a.new_max_pages;
  p.page_size = a.page_size;
  p.keep = a.keep;
  p.first = a.first;
  p.recent = a.recent;
  p.chunks = (a.keep + kChunk - 1) / kChunk;
  p.by_heads = make_fast_div(a.kv_heads);
  p.by_chunks = make_fast_div(p.chunks);
  p.kept = a.kept;
  p.new_seqlens = a.new_seqlens;
  p.new_weights = a.new_weights;
  p.page_ok = page_ok;
  p.bitmap_words = std::max(1, std::min((a.num_pages + 31) / 32, kMostBitmapWords));
  p.status = status;
  const cudaError_t e = launch_select(p, sms, stream);
  if (e != cudaSuccess) return e;
  const int jobs = a.batch * p.chunks * a.kv_heads;
  const dim3 grid(std::min(jobs, sms * 4));
  return a.head_dim == 128 ? launch_after(fp8_evict_move_kernel<128>, grid, dim3(kThreads), 0, stream, p, jobs)
                           : launch_after(fp8_evict_move_kernel<64>, grid, dim3(kThreads), 0, stream, p, jobs);
}

}  // namespace jfa
