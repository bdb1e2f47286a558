// Filling the bf16 paged cache and keeping what was accepted of its drafts
// (the attention in between: decode_tree.cu).
//
// Append: a token's q and k turn by its position, k and v go to its page. In
// 16-byte pieces of a head, piece by piece and lane by lane: for pairs (j, j + rot / 2)
// the other half of a pair lies rot / 16 lanes on, and moves by a shuffle; a lane
// keeps its columns, and so its cosines and sines, for all heads of a token.
//   x' = x cos - y sin,  y' = y cos + x sin   in fp32, rounded to bf16 once.
// Bound by HBM: 4 d (Hq + 2 Hkv) + 4 rot bytes a token. 16 prompts of 61-8192 tokens, 32 heads
// on 8 of 128: 257 us, 95% of the copy rate; one token a sequence is a chain of four loads, 3.5 us.
//
// Accept: the accepted drafts' K and V rows move down to the places behind the
// earlier tokens. A thread owns 16 bytes of every row, so what it overwrites it has read
// itself. Latency: a chain of lengths, indexes, pages, rows (3.3 us; 512 sequences of up to 17
// rows 7.0, two thirds of the copy rate).
#include <algorithm>

#include "fp8_cache.cuh"

namespace jfa {

namespace {

constexpr int kReportThreads = 256;

// ------------------------------------------------------------------ append with rotation

constexpr int kAppendWarps = 4;  // warps of a block, which share one token's heads
constexpr int kAppendBatch = 6;  // pieces that a lane has in flight

struct AppendRopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* offsets;
  const int32_t* positions;
  const float* cos_table;
  const float* sin_table;
  __nv_bfloat16* q_out;
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  const int32_t* page_table;
  const int32_t* seqlens;
  int64_t qs, ks, vs;
  int32_t batch, hq, hkv, rot, table_rows, num_pages, max_pages, total_new;
  int32_t share;  // warps that share a token: kAppendWarps, or 1
  FastDiv page;
  int32_t* status;
};

__device__ __forceinline__ bool new_range_ok(int b, int o0, int o1, int L, int total, int64_t cap) {
  return o0 >= 0 && o1 >= o0 && o1 <= total && L >= o1 - o0 && L <= cap && (b > 0 || o0 == 0);
}

// The last sequence whose first row is not above `row`, 32 bounds looked at together, first far apart.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int batch, int row) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0, n = batch;
  while (n > 1) {
    const uint32_t step = (n + 31) >> 5;
    const bool in = lane * step < n && offsets[lo + lane * step] <= row;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const uint32_t k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return static_cast<int>(lo);
}

// One more block checks the whole call and writes the status block; the others pass over what is
// wrong. A thread a sequence, the pages of those with many new ones by warps.
__device__ void append_rope_report(const AppendRopeParams& p, int64_t cap) {
  __shared__ int32_t s_left, s_b[32 * kAppendWarps], s_lo[32 * kAppendWarps], s_hi[32 * kAppendWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  auto check = [&](int b, int i) {
    bad |= static_cast<uint32_t>(p.page_table[static_cast<int64_t>(b) * p.max_pages + i]) >=
           static_cast<uint32_t>(p.num_pages);
  };
  if (p.positions && p.rot > 0) {
    const int used = min(p.offsets[p.batch], p.total_new);
#pragma unroll 4
    for (int i = tid; i < used; i += blockDim.x)
      bad |= static_cast<uint32_t>(p.positions[i]) >= static_cast<uint32_t>(p.table_rows);
  }
  for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
    if (tid == 0) s_left = 0;
    __syncthreads();
    const int b = b0 + tid;
    if (b < p.batch) {
      const int o0 = p.offsets[b], o1 = p.offsets[b + 1], L = p.seqlens[b];
      if (!new_range_ok(b, o0, o1, L, p.total_new, cap)) {
        bad = true;
      } else if (o1 > o0) {
        bad |= !p.positions && p.rot > 0 && L > p.table_rows;
        const int lo = fast_div(L - (o1 - o0), p.page), hi = fast_div(L - 1, p.page);
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
    for (int j = tid >> 5; j < s_left; j += kAppendWarps) {
      const int last = s_hi[j];
#pragma unroll 16
      for (int i = s_lo[j] + lane; i <= last; i += 32) check(s_b[j], i);
    }
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  if (tid < static_cast<int>(kStatusBytes / 4))
    p.status[tid] = !bad ? 0 : (tid == 0 ? JFA_ERR_BAD_INPUT : (tid == 1 ? kSiteAppendRope : 0));
}

// A warp a token, or a block.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kAppendWarps) append_rope_kernel(const AppendRopeParams p) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a head, heads of a warp
  const int64_t cap = static_cast<int64_t>(p.num_pages ? p.max_pages : 0) * p.page.d;
  if (blockIdx.x == gridDim.x - 1) {
    append_rope_report(p, cap);
    return;
  }
  const int lane = threadIdx.x & 31, share = p.share;
  const int warp = (threadIdx.x >> 5) & (share - 1);  // among those of its token
  const int row = (blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) / share;
  if (row >= p.total_new) return;
  const int b = sequence_of(p.offsets, p.batch, row);
  const int o0 = p.offsets[b], o1 = p.offsets[b + 1], L = p.seqlens[b];
  if (row < o0 || row >= o1 || !new_range_ok(b, o0, o1, L, p.total_new, cap)) return;
  const int at = L - o1 + row;
  const int turn = p.rot == 0 ? 0 : (p.positions ? p.positions[row] : at);
  const int slot_page = fast_div(at, p.page);
  const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + slot_page];
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) return;
  if (p.rot > 0 && static_cast<uint32_t>(turn) >= static_cast<uint32_t>(p.table_rows)) return;
  const int64_t cell = static_cast<int64_t>(page) * p.page.d + (at - slot_page * static_cast<int>(p.page.d));

  const int col = (lane % kLanes) * 8, half = p.rot >> 1;
  const bool turns = col < p.rot;
  // pairs (j, j + half): this lane's eight columns and their partner lane; neighbours: four pairs of its own
  const bool upper = col >= half;
  const int partner = !turns ? lane : (upper ? lane - half / 8 : lane + half / 8);
  float c[INTERLEAVED ? 4 : 8], s[INTERLEAVED ? 4 : 8];
  if (turns) {
    const int64_t first = static_cast<int64_t>(turn) * half + (INTERLEAVED ? col >> 1 : (upper ? col - half : col));
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 1 : 2); ++i) {
      const float4 cv = *reinterpret_cast<const float4*>(p.cos_table + first + 4 * i);
      const float4 sv = *reinterpret_cast<const float4*>(p.sin_table + first + 4 * i);
      c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
      s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
    }
  }
  const int hq = p.q ? p.hq : 0, heads = hq + 2 * p.hkv;
  const __nv_bfloat16* src_q = p.q + row * p.qs + col;
  const __nv_bfloat16* src_k = p.k + row * p.ks + col;
  const __nv_bfloat16* src_v = p.v + row * p.vs + col;
  for (int h0 = warp * kPer; h0 < heads; h0 += share * kPer * kAppendBatch) {
    uint4 x[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int h = h0 + i * share * kPer + lane / kLanes;
      if (h < hq)
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src_q + h * D));
      else if (h < hq + p.hkv)
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src_k + (h - hq) * D));
      else if (h < heads)
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src_v + (h - hq - p.hkv) * D));
      else
        x[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int h = h0 + i * share * kPer + lane / kLanes;
      uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      if (INTERLEAVED) {
        if (turns && h < hq + p.hkv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = ptx::bf16lo(w[e]), d = ptx::bf16hi(w[e]);
            w[e] = ptx::pack_bf16(a * c[e] - d * s[e], d * c[e] + a * s[e]);
          }
        }
      } else {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __shfl_sync(0xffffffffu, w[e], partner);
        if (turns && h < hq + p.hkv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sl = upper ? s[2 * e] : -s[2 * e], sh = upper ? s[2 * e + 1] : -s[2 * e + 1];
            w[e] = ptx::pack_bf16(ptx::bf16lo(w[e]) * c[2 * e] + ptx::bf16lo(y[e]) * sl,
                                  ptx::bf16hi(w[e]) * c[2 * e + 1] + ptx::bf16hi(y[e]) * sh);
          }
        }
      }
      __nv_bfloat16* dst = nullptr;
      if (h < hq)
        dst = p.q_out + (static_cast<int64_t>(row) * p.hq + h) * D + col;
      else if (h < hq + p.hkv)
        dst = p.kc + (cell * p.hkv + h - hq) * D + col;
      else if (h < heads)
        dst = p.vc + (cell * p.hkv + h - hq - p.hkv) * D + col;
      if (dst) ptx::st_v4(dst, w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------------ accept

struct AcceptParams {
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* offsets;
  const int32_t* accepted;
  const int32_t* counts;
  int32_t batch, num_pages, max_pages, width;
  FastDiv page;
  int32_t* new_seqlens;
  int32_t* status;
};

constexpr int kAcceptAhead = 8;  // rows that a thread has in flight

// The row of the cache that holds position t of sequence b, or -1.
__device__ __forceinline__ int64_t cache_row(const AcceptParams& p, int b, int t) {
  const int pg = fast_div(t, p.page);
  const int page = p.page_table[static_cast<int64_t>(b) * p.max_pages + pg];
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) return -1;
  return static_cast<int64_t>(page) * p.page.d + (t - pg * static_cast<int>(p.page.d));
}

// The length before the drafts and their number; false where lengths or offsets are out of range.
__device__ __forceinline__ bool accept_range(const AcceptParams& p, int b, int64_t cap, int& C, int& n, int& L) {
  const int o0 = p.offsets[b], o1 = p.offsets[b + 1];
  L = p.seqlens[b];
  n = o1 - o0;
  C = L - n;
  return new_range_ok(b, o0, o1, L, 0x7fffffff, cap);
}
// One block checks the whole call, writes the new lengths and the status block: a thread a sequence,
// its entries eight at a time (512 sequences of up to 17 entries, one after the other: 27 us).
__device__ void accept_report(const AcceptParams& p, int64_t cap) {
  constexpr int kAhead = 8;
  bool bad = false;
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    int C, n, L;
    const bool ok = accept_range(p, b, cap, C, n, L);
    const int count = p.counts[b];
    bool good = ok && count >= 0 && count <= p.width && count <= n;
    if (good) {
      const int32_t* list = p.accepted + static_cast<int64_t>(b) * p.width;
      const int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
      for (int k0 = 0; k0 < count; k0 += kAhead) {
        int j[kAhead], from[kAhead], to[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) j[e] = list[min(k0 + e, count - 1)];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const bool in = j[e] >= 0 && j[e] < n;
          good &= in;
          from[e] = row[fast_div(C + (in ? j[e] : 0), p.page)];
          to[e] = row[fast_div(C + min(k0 + e, count - 1), p.page)];
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          good &= static_cast<uint32_t>(from[e]) < static_cast<uint32_t>(p.num_pages) &&
                  static_cast<uint32_t>(to[e]) < static_cast<uint32_t>(p.num_pages);
      }
    }
    p.new_seqlens[b] = !ok ? L : (good ? C + count : C);
    bad |= !good;
  }
  bad = __syncthreads_or(bad);
  for (int i = threadIdx.x; i < static_cast<int>(kStatusBytes / 4); i += blockDim.x)
    p.status[i] = !bad ? 0 : (i == 0 ? JFA_ERR_BAD_INPUT : (i == 1 ? kSiteAccept : 0));
}

// A block 256 pieces of a sequence's rows, K's before V's (a block a head of each: 24 us for 512
// sequences, mostly the same chain of loads in 8192 blocks).
__global__ void __launch_bounds__(kReportThreads) accept_kernel(const AcceptParams p, int pieces) {
  __shared__ int64_t s_from[kTreeMaxNodes], s_to[kTreeMaxNodes];
  const int64_t cap = static_cast<int64_t>(p.num_pages ? p.max_pages : 0) * p.page.d;
  const int b = blockIdx.x;
  if (b == p.batch) {
    if (blockIdx.y == 0) accept_report(p, cap);
    return;
  }
  int C, n, L;
  if (!accept_range(p, b, cap, C, n, L)) return;
  const int count = p.counts[b];
  if (count < 1 || count > p.width || count > n) return;
  bool good = true, rising = true;
  if (threadIdx.x < count) {
    const int k = threadIdx.x;
    const int32_t* list = p.accepted + static_cast<int64_t>(b) * p.width;
    const int j = list[k], before = k ? list[k - 1] : -1;
    good = j >= 0 && j < n;
    rising = j > before;
    s_from[k] = good ? cache_row(p, b, C + j) : -1;
    s_to[k] = cache_row(p, b, C + k);
    good = s_from[k] >= 0 && s_to[k] >= 0;
  }
  if (!__syncthreads_and(good)) return;
  rising = __syncthreads_and(rising);
  const int piece = blockIdx.y * kReportThreads + threadIdx.x;
  if (piece >= 2 * pieces) return;
  uint4* c = reinterpret_cast<uint4*>(piece < pieces ? p.kc : p.vc) + (piece < pieces ? piece : piece - pieces);
  if (rising) {  // a place lies at or before its source, and later sources behind both: in order, a few together
    for (int k0 = 0; k0 < count; k0 += kAcceptAhead) {
      uint4 x[kAcceptAhead];
#pragma unroll
      for (int e = 0; e < kAcceptAhead; ++e) x[e] = c[s_from[min(k0 + e, count - 1)] * pieces];
#pragma unroll
      for (int e = 0; e < kAcceptAhead; ++e)
        if (k0 + e < count && s_from[k0 + e] != s_to[k0 + e]) c[s_to[k0 + e] * pieces] = x[e];
    }
  } else {
    // Any order, an index more than once: all is read before any is written. The rows lie in local memory: falling
    // paths take 10.6 us where rising ones take 6.9 (512 sequences of up to 17 rows), 47.5 against 22.8 (of 64).
    uint4 x[kTreeMaxNodes];
    for (int k = 0; k < count; ++k) x[k] = c[s_from[k] * pieces];
    for (int k = 0; k < count; ++k) c[s_to[k] * pieces] = x[k];
  }
}

}  // namespace

cudaError_t launch_cache_append_rope(const jfa_cache_append_rope_args& a, int32_t* status, cudaStream_t stream) {
  AppendRopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.offsets = a.new_offsets;
  p.positions = a.positions;
  p.cos_table = a.cos_table;
  p.sin_table = a.sin_table;
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.kc = static_cast<__nv_bfloat16*>(a.k_cache);
  p.vc = static_cast<__nv_bfloat16*>(a.v_cache);
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.qs = a.q_stride;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.batch = a.batch;
  p.hq = a.q_heads;
  p.hkv = a.kv_heads;
  p.rot = a.rot_dim;
  p.table_rows = a.table_rows;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.total_new = a.total_new;
  p.page = make_fast_div(a.page_size);
  p.status = status;
  // Few tokens leave the device empty, and a block each shortens their chain; many keep it full with a warp
  // each, which looks its sequence, page and angles up once for all heads. 32 heads on 8 of 128: one token 3.4 us
  // (a warp 6.4), 512 sequences of one 5.0 (7.4), 2048 of one 19.0 (13.8), 16 prompts of 61-8192 291 (257),
  // the same of head_dim 64 217 (140).
  p.share = a.total_new <= 1024 ? kAppendWarps : 1;
  const int per_block = kAppendWarps / p.share;
  const int grid = (a.total_new + per_block - 1) / per_block + 1;
  if (a.head_dim == 128) {
    if (a.interleaved)
      append_rope_kernel<128, true><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
    else
      append_rope_kernel<128, false><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  } else {
    if (a.interleaved)
      append_rope_kernel<64, true><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
    else
      append_rope_kernel<64, false><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_accept(const jfa_cache_accept_args& a, int32_t* status, cudaStream_t stream) {
  AcceptParams p{};
  p.kc = static_cast<__nv_bfloat16*>(a.k_cache);
  p.vc = static_cast<__nv_bfloat16*>(a.v_cache);
  p.page_table = a.page_table;
  p.seqlens = a.seqlens_k;
  p.offsets = a.q_offsets;
  p.accepted = a.accepted;
  p.counts = a.counts;
  p.batch = a.batch;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.width = a.width;
  p.page = make_fast_div(a.page_size);
  p.new_seqlens = a.new_seqlens;
  p.status = status;
  const int pieces = a.kv_heads * a.head_dim / 8;  // 16-byte pieces of a row
  const dim3 grid(a.batch + 1, (2 * pieces + kReportThreads - 1) / kReportThreads);
  accept_kernel<<<grid, kReportThreads, 0, stream>>>(p, pieces);
  return cudaGetLastError();
}

}  // namespace jfa
