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
// Both kernels that write codes give 128 consecutive positions of one head's K
// or V to a block of threads: whole scale blocks (a power of two up to 128), the
// values held in registers between the amax and the encoding, so every byte
// is read once.
#include <cuda_fp16.h>

#include "fp8_cache.cuh"

namespace jfa {

constexpr int kChunk = 128;    // positions of one block of threads
constexpr int kThreads = 256;

// ------------------------------------------------------------------ append

struct Fp8AppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* new_offsets;
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  int32_t batch, max_pages, page_size, total_new, max_new, chunks;
  float* weights;
  int32_t* status;
};

// e4m3 codes of eight values divided by s. A power of two (every scale that
// this file writes) divides exactly by a multiplication; other scales take the
// rounded quotient.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s) {
  float y[8];
  if ((__float_as_uint(s) & 0x7FFFFFu) == 0) {
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
  }
  return make_uint2(f32x2_to_e4m3x2(y[0], y[1]) | (f32x2_to_e4m3x2(y[2], y[3]) << 16),
                    f32x2_to_e4m3x2(y[4], y[5]) | (f32x2_to_e4m3x2(y[6], y[7]) << 16));
}

// The values of eight codes at scale s.
__device__ __forceinline__ void decode8(uint2 codes, float s, float (&x)[8]) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16(w[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[4 * i] = a.x * s;
    x[4 * i + 1] = a.y * s;
    x[4 * i + 2] = b.x * s;
    x[4 * i + 3] = b.y * s;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) fp8_append_kernel(const Fp8AppendParams p) {
  constexpr int kLanes = D / 8;              // threads of a row, 8 values each
  constexpr int kRowsPerPass = kThreads / kLanes;
  constexpr int kPasses = kChunk / kRowsPerPass;
  __shared__ int32_t s_row[kChunk];          // cache row of each position, -1: nothing there to touch
  __shared__ uint32_t s_amax[kChunk];        // per scale block, the bits of a non-negative float
  __shared__ float s_new[kChunk], s_old[kChunk];

  wait_prior_grid();  // the cleared status block
  const int b = blockIdx.x / p.chunks, ci = blockIdx.x % p.chunks;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int hkv = p.c.hkv;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int o0 = p.new_offsets[b], o1 = p.new_offsets[b + 1], L = p.seqlens[b];
  // offsets rise from 0 to total_new, and the new tokens are part of the length
  if (o0 < 0 || o1 < o0 || o1 > p.total_new || o1 - o0 > p.max_new || L < o1 - o0 || L > cap ||
      (b == 0 && o0 != 0) || (b == p.batch - 1 && o1 != p.total_new)) {
    if (threadIdx.x == 0) flag_bad_cache(p.status, kSiteFp8Append);
    return;
  }
  const int f = L - (o1 - o0);                 // first new position
  const int p0 = ((f / kChunk) + ci) * kChunk;  // this block's positions: p0 .. p0 + 127
  if (o1 == o0 || p0 >= L) return;
  const int bs = p.c.block_shift;
  const int old0 = (f >> bs) << bs;            // older tokens of f's block: old0 .. f - 1

  const int tid = threadIdx.x;
  if (tid < kChunk) {
    const int pos = p0 + tid;
    int row = -1;
    if (pos >= old0 && pos < L) {
      const int pg = fast_div(pos, p.c.page);
      const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pg];
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.c.num_pages))
        row = page * p.page_size + (pos - pg * p.page_size);
      else
        flag_bad_cache(p.status, kSiteFp8Append);
    }
    s_row[tid] = row;
    s_amax[tid] = 0;
    if (p.weights && !is_v && pos >= f && pos < L)
      p.weights[(static_cast<int64_t>(b) * hkv + h) * cap + pos] = 0.f;
  }
  const int sub = tid % kLanes, r0 = tid / kLanes;
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + static_cast<int64_t>(h) * D + 8 * sub;
  uint4 raw[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int pos = p0 + k * kRowsPerPass + r0;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (pos >= f && pos < L)
      raw[k] = __ldg(reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(o0) + pos - f) * hkv * D));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // infinities and NaN do not set the scale
      const float x0 = fabsf(ptx::bf16lo(w[i])), x1 = fabsf(ptx::bf16hi(w[i]));
      a = fmaxf(a, fmaxf(x0 < INFINITY ? x0 : 0.f, x1 < INFINITY ? x1 : 0.f));
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (sub == 0 && a > 0.f) atomicMax(&s_amax[(k * kRowsPerPass + r0) >> bs], __float_as_uint(a));
  }
  __syncthreads();
  float* scales = is_v ? p.c.vs : p.c.ks;
  if (tid < (kChunk >> bs)) {
    const int start = p0 + (tid << bs);
    const int pos = max(start, f);  // the block's first new position, if it has one
    if (pos < min(L, start + (1 << bs)) && s_row[pos - p0] >= 0) {
      float s = e4m3_block_scale(__uint_as_float(s_amax[tid]));
      float* cell = scales + static_cast<int64_t>(s_row[pos - p0] >> bs) * hkv + h;
      const float old = start < f ? *cell : 0.f;
      s = fmaxf(s, old);
      s_old[tid] = start < f ? old : s;
      s_new[tid] = s;
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
    uint2* dst = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(row) * hkv * D);
    const float s = s_new[t >> bs];
    float x[8];
    if (pos >= f) {
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = ptx::bf16lo(w[i]);
        x[2 * i + 1] = ptx::bf16hi(w[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fabsf(x[i]) < INFINITY ? x[i] : __int_as_float(0x7fffffff);
      *dst = encode8(x, s);
    } else if (s_old[t >> bs] != s) {  // an older token of a block whose scale has grown
      decode8(*dst, s_old[t >> bs], x);
      *dst = encode8(x, s);
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
  // n consecutive positions touch at most (n + 126) / 128 + 1 chunks
  p.chunks = static_cast<int32_t>((static_cast<int64_t>(a.max_new) + kChunk - 2) / kChunk + 1);
  p.weights = a.weights;
  p.status = status;
  const dim3 grid(static_cast<uint32_t>(p.batch) * static_cast<uint32_t>(p.chunks),
                  static_cast<uint32_t>(a.kv_heads) * 2);
  return a.head_dim == 128 ? launch_after(fp8_append_kernel<128>, grid, dim3(kThreads), 0, stream, p)
                           : launch_after(fp8_append_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

// ------------------------------------------------------------------ evict

struct Fp8EvictParams {
  Fp8CacheView c;
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* new_table;
  const float* weights;
  int32_t batch, max_pages, new_max_pages, page_size, keep, first, recent, chunks;
  int32_t* kept;         // [B, hkv, keep]
  int32_t* new_seqlens;  // [B]
  float* new_weights;    // [B, hkv, new_max_pages * page_size]
  uint32_t* page_state;  // [num_pages]: bit 31 = read from, below: how often it is written to
  int32_t* status;
};

constexpr int kSelThreads = 1024;
constexpr uint32_t kPageRead = 0x80000000u;

__global__ void __launch_bounds__(kThreads) fp8_evict_init_kernel(int32_t* status, uint32_t* page_state, int n) {
  allow_next_grid();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i < kStatusBytes / 4) status[i] = 0;
  if (i < n) page_state[i] = 0;
}

// Order of the weights as unsigned numbers; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w == w ? w + 0.f : -INFINITY);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the threads before this one (exclusive); *total gets the whole sum.
__device__ __forceinline__ int block_exclusive_sum(int x, int32_t* warp_sum, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) y += z;
  }
  __syncthreads();  // warp_sum may still be read from an earlier call
  if (lane == 31) warp_sum[warp] = y;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    const int s = warp_sum[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  return before + y - x;
}

// One block per (sequence, KV head): what stays, in order.
__global__ void __launch_bounds__(kSelThreads, 1) fp8_evict_select_kernel(const Fp8EvictParams p) {
  __shared__ int32_t hist[2048];
  __shared__ int32_t warp_sum[32];
  __shared__ uint32_t s_prefix;
  __shared__ int32_t s_need;
  wait_prior_grid();
  allow_next_grid();
  const int b = blockIdx.x / p.c.hkv, h = blockIdx.x % p.c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t new_cap = static_cast<int64_t>(p.new_max_pages) * p.page_size;
  int L = p.seqlens[b];
  if (L < 0 || L > cap || (L > 0 && p.c.num_pages == 0)) {
    if (tid == 0) flag_bad_cache(p.status, kSiteFp8Evict);
    L = 0;
  }
  const int n = min(L, p.keep);
  const float* w = p.weights + static_cast<int64_t>(blockIdx.x) * cap;
  int32_t* kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.keep;
  float* nw = p.new_weights + static_cast<int64_t>(blockIdx.x) * new_cap;
  if (h == 0) {
    if (tid == 0) p.new_seqlens[b] = n;
    // pages read by this sequence and pages it will write
    const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    const int32_t* nt = p.new_table + static_cast<int64_t>(b) * p.new_max_pages;
    const int used = L > 0 ? fast_div(L - 1, p.c.page) + 1 : 0, fresh = n > 0 ? fast_div(n - 1, p.c.page) + 1 : 0;
    for (int i = tid; i < used; i += kSelThreads) {
      const uint32_t pg = static_cast<uint32_t>(pt[i]);
      if (pg < static_cast<uint32_t>(p.c.num_pages)) atomicOr(p.page_state + pg, kPageRead);
    }
    for (int i = tid; i < fresh; i += kSelThreads) {
      const uint32_t pg = static_cast<uint32_t>(nt[i]);
      if (pg < static_cast<uint32_t>(p.c.num_pages)) atomicAdd(p.page_state + pg, 1u);
    }
  }
  for (int64_t j = n + tid; j < p.keep; j += kSelThreads) kept[j] = -1;
  for (int64_t j = n + tid; j < new_cap; j += kSelThreads) nw[j] = 0.f;
  if (L <= p.keep) {
    for (int j = tid; j < n; j += kSelThreads) {
      kept[j] = j;
      nw[j] = w[j];
    }
    return;
  }
  const int c0 = p.first, c1 = L - p.recent;           // candidates
  const int want = p.keep - p.first - p.recent;        // of which this many stay, 0 <= want < c1 - c0
  // The want-th largest key, digit by digit (11, 11 and 10 bits from the top).
  uint32_t prefix = 0;
  int need = want;  // how many keys with the prefix found so far stay
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);  // the prefix's bits end here
      for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t0 = c0 + warp * 32; t0 < c1; t0 += kSelThreads) {
        uint32_t d = 2048;  // no digit
        if (t0 + lane < c1) {
          const uint32_t k = weight_key(w[t0 + lane]);
          if (pass == 0 || (k >> above) == prefix) d = (k >> shift) & mask;
        }
        // equal digits of a warp count once: caches of mostly equal weights are common
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (d < 2048 && lane == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
      }
      __syncthreads();
      // bins from the top: thread t holds bins 2047 - 2 t and 2046 - 2 t
      const int h0 = hist[2047 - 2 * tid], h1 = hist[2046 - 2 * tid];
      int all;
      const int before = block_exclusive_sum(h0 + h1, warp_sum, &all);
      if (before < need && before + h0 + h1 >= need) {
        const bool upper = before + h0 >= need;
        const uint32_t d = upper ? 2047 - 2 * tid : 2046 - 2 * tid;
        s_prefix = pass == 2 ? (prefix << 10) | d : (prefix << 11) | d;
        s_need = need - before - (upper ? 0 : h0);
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // keys above `prefix` stay, and the first `need` that equal it
  for (int j = tid; j < p.first; j += kSelThreads) {
    kept[j] = j;
    nw[j] = w[j];
  }
  for (int j = tid; j < p.recent; j += kSelThreads) {
    kept[p.keep - p.recent + j] = c1 + j;
    nw[p.keep - p.recent + j] = w[c1 + j];
  }
  if (want == 0) return;
  const int per_warp = (c1 - c0 + kSelThreads - 1) / kSelThreads * 32;  // a run of candidates for each warp
  const int lo = min(c0 + warp * per_warp, c1), hi = min(lo + per_warp, c1);
  int gt = 0, eq = 0;
  for (int t = lo; t < hi; t += 32) {
    const uint32_t k = t + lane < hi ? weight_key(w[t + lane]) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, t + lane < hi && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, t + lane < hi && k == prefix));
  }
  int all;
  int gt0 = block_exclusive_sum(lane == 0 ? gt : 0, warp_sum, &all);
  int eq0 = block_exclusive_sum(lane == 0 ? eq : 0, warp_sum, &all);
  gt0 = __shfl_sync(0xffffffffu, gt0, 0);
  eq0 = __shfl_sync(0xffffffffu, eq0, 0);
  const uint32_t below = (1u << lane) - 1;
  for (int t = lo; t < hi; t += 32) {
    const float x = t + lane < hi ? w[t + lane] : 0.f;
    const uint32_t k = weight_key(x);
    const uint32_t mg = __ballot_sync(0xffffffffu, t + lane < hi && k > prefix);
    const uint32_t me = __ballot_sync(0xffffffffu, t + lane < hi && k == prefix);
    const int eq_rank = eq0 + __popc(me & below);
    const bool mine = ((mg >> lane) & 1) || (((me >> lane) & 1) && eq_rank < need);
    if (mine) {
      const int j = p.first + gt0 + __popc(mg & below) + min(eq_rank, need);
      kept[j] = t + lane;
      nw[j] = x;
    }
    gt0 += __popc(mg);
    eq0 += __popc(me);
  }
}

// Moves the kept rows of 128 new positions of one head's K or V.
template <int D>
__global__ void __launch_bounds__(kThreads) fp8_evict_move_kernel(const Fp8EvictParams p) {
  constexpr int kLanes = D / 16;             // threads of a row, 16 codes each
  constexpr int kRowsPerPass = kThreads / kLanes;
  constexpr int kPasses = kChunk / kRowsPerPass;
  __shared__ int32_t s_src[kChunk], s_dst[kChunk];  // cache rows, -1: none
  __shared__ uint32_t s_amax[kChunk];
  __shared__ float s_new[kChunk];

  wait_prior_grid();
  const int b = blockIdx.x / p.chunks, j0 = (blockIdx.x % p.chunks) * kChunk;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int hkv = p.c.hkv, bs = p.c.block_shift, tid = threadIdx.x;
  const int n = p.new_seqlens[b];
  if (j0 >= n) return;
  if (tid < kChunk) {
    const int j = j0 + tid;
    int src = -1, dst = -1;
    if (j < n) {
      const int t = p.kept[(static_cast<int64_t>(b) * hkv + h) * p.keep + j];
      const int pg = fast_div(t, p.c.page), npg = fast_div(j, p.c.page);
      const uint32_t page = static_cast<uint32_t>(p.page_table[static_cast<int64_t>(b) * p.max_pages + pg]);
      const uint32_t fresh = static_cast<uint32_t>(p.new_table[static_cast<int64_t>(b) * p.new_max_pages + npg]);
      const uint32_t pages = static_cast<uint32_t>(p.c.num_pages);
      if (page < pages) src = static_cast<int>(page) * p.page_size + (t - pg * p.page_size);
      // a page that some sequence still reads, or that is given out twice, is not written
      if (fresh < pages && p.page_state[fresh] == 1u) dst = static_cast<int>(fresh) * p.page_size + (j - npg * p.page_size);
      if (src < 0 || dst < 0) flag_bad_cache(p.status, kSiteFp8Evict);
    }
    s_src[tid] = src;
    s_dst[tid] = dst;
    s_amax[tid] = 0;
  }
  __syncthreads();
  const int sub = tid % kLanes, r0 = tid / kLanes;
  uint8_t* codes = (is_v ? p.c.vc : p.c.kc) + static_cast<int64_t>(h) * D + 16 * sub;
  float* scales = (is_v ? p.c.vs : p.c.ks) + h;
  uint4 raw[kPasses];
  float sc[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int src = s_src[k * kRowsPerPass + r0];
    raw[k] = make_uint4(0, 0, 0, 0);  // a token whose page is missing becomes zeros
    sc[k] = 0.f;
    if (src >= 0) {
      raw[k] = *reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(src) * hkv * D);
      sc[k] = scales[static_cast<int64_t>(src >> bs) * hkv];
    }
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    uint32_t top = 0;  // largest magnitude code, byte by byte, without NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = w[i] & 0x7F7F7F7Fu;
      const uint32_t nan = ((m + 0x01010101u) & 0x80808080u) >> 7;
      top = __vmaxu4(top, m & ~(nan * 0xFFu));
    }
    top = max(max(top & 0xFFu, (top >> 8) & 0xFFu), max((top >> 16) & 0xFFu, top >> 24));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (sub == 0 && top) {
      const uint32_t f16 = e4m3x2_to_f16x2(static_cast<uint16_t>(top));
      const float a = fminf(__low2float(*reinterpret_cast<const __half2*>(&f16)) * sc[k], 3.4028234e38f);
      atomicMax(&s_amax[(k * kRowsPerPass + r0) >> bs], __float_as_uint(a));
    }
  }
  __syncthreads();
  if (tid < (kChunk >> bs)) {
    const float s = e4m3_block_scale(__uint_as_float(s_amax[tid]));
    s_new[tid] = s;
    const int dst = s_dst[tid << bs];
    if (dst >= 0) scales[static_cast<int64_t>(dst >> bs) * hkv] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int t = k * kRowsPerPass + r0;
    const int dst = s_dst[t];
    if (dst < 0) continue;
    const float s = s_new[t >> bs];
    uint4 out = raw[k];
    if (s != sc[k]) {
      float x[8];
      decode8(make_uint2(raw[k].x, raw[k].y), sc[k], x);
      const uint2 lo = encode8(x, s);
      decode8(make_uint2(raw[k].z, raw[k].w), sc[k], x);
      const uint2 hi = encode8(x, s);
      out = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(dst) * hkv * D) = out;
  }
}

cudaError_t launch_cache_evict_fp8(const jfa_cache_evict_fp8_args& a, uint32_t* page_state, int32_t* status,
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
  p.kept = a.kept;
  p.new_seqlens = a.new_seqlens;
  p.new_weights = a.new_weights;
  p.page_state = page_state;
  p.status = status;
  const int words = a.num_pages > static_cast<int>(kStatusBytes / 4) ? a.num_pages : static_cast<int>(kStatusBytes / 4);
  fp8_evict_init_kernel<<<(words + kThreads - 1) / kThreads, kThreads, 0, stream>>>(status, page_state, a.num_pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(fp8_evict_select_kernel, dim3(static_cast<uint32_t>(a.batch) * a.kv_heads), dim3(kSelThreads), 0,
                   stream, p);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(a.batch) * static_cast<uint32_t>(p.chunks), static_cast<uint32_t>(a.kv_heads) * 2);
  return a.head_dim == 128 ? launch_after(fp8_evict_move_kernel<128>, grid, dim3(kThreads), 0, stream, p)
                           : launch_after(fp8_evict_move_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace jfa
