// cache.cu -- the paged key/value cache of a speculative step: the plan
// (blocks granted and slots mapped from the lengths, dspark_cache_plan) and
// the write of new keys and values (dspark_kv_write).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#define DSPARK_TU 10  // this file's number in the checked build's site codes
#include "common.cuh"

namespace dspark {

// --------------------------------------------------------------- the plan
// A CTA plans `group` consecutive requests and, for long prompts, one range
// of their tokens (blockIdx.y).  The blocks granted before its group are the
// sum of every earlier request's need: each CTA takes that sum from the
// lengths itself (8 bytes a request, in L2 after the first CTA), so the plan
// is one launch without a wait between CTAs, and its work grows with the
// square of the requests: 0.07 ms for 2^16 of them, 4.3 ms for the most,
// DSPARK_MAX_PLANNED, over an hour for the 2^30 that the arrays' sizes alone
// would allow.  A batch's time is a chain of loads and two block scans: 4 us
// for 256 chains of 6, 6 us for 1,023 trees of 64 nodes, 8 us for 96 prompts
// of up to 8,192 tokens.
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanCells = 1024;   // most (request, token) pairs of a CTA
constexpr int kPlanMaxGroup = kPlanThreads;  // one thread takes one request's need

struct PlanParams {
  const int32_t* ctx;
  const int32_t* added;
  int B, max_new, page;
  int32_t* table;
  int64_t table_ld;
  int max_blocks;
  const int32_t* free_blocks;
  int max_free;
  const int32_t* n_free;
  const int32_t* parents;
  int32_t* slots;
  int32_t* positions;
  uint64_t* mask;
  int32_t* taken;
  int32_t* status;
  int group, span;  // requests per CTA (at most kPlanMaxGroup); tokens of each per CTA
};

struct Need {
  int held, need;
  bool valid;
};

__device__ __forceinline__ Need request_need(const PlanParams& p, int b) {
  const int ctx = p.ctx[b], add = p.added[b];
  Need n;
  n.held = n.need = 0;
  n.valid = ctx >= 0 && add >= 0 && add <= p.max_new;
  if (n.valid) {
    const uint32_t page = (uint32_t)p.page, sum = (uint32_t)ctx + (uint32_t)add;  // < 2^32
    const uint32_t end = sum / page + (sum % page != 0u);
    n.held = (int)((uint32_t)ctx / page + ((uint32_t)ctx % page != 0u));
    n.valid = end <= (uint32_t)p.max_blocks;  // so sum <= max_blocks * page < 2^31
    n.need = n.valid ? (int)end - n.held : 0;
  }
  return n;
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams p) {
  __shared__ uint64_t scratch[32];
  __shared__ int64_t s_off[kPlanMaxGroup];  // the group's exclusive offsets; -1: refused
  __shared__ int s_held[kPlanMaxGroup];
  __shared__ int s_need[kPlanMaxGroup];
  __shared__ uint32_t s_bad[kPlanMaxGroup];  // a parent out of range
  __shared__ int s_parent[kPlanCells];
  const int tid = threadIdx.x;
  const int first = blockIdx.x * p.group;
  const int n = min(p.group, p.B - first);

  uint64_t before = 0;
  for (int b = tid; b < first; b += kPlanThreads) before += (uint64_t)request_need(p, b).need;
  const int64_t base = (int64_t)block_reduce(before, OpAddU64(), scratch);

  int64_t n_free = p.max_free;
  if (p.n_free) n_free = max(0, min(p.max_free, *p.n_free));

  Need mine = {0, 0, false};
  if (tid < n) mine = request_need(p, first + tid);
  uint64_t total;
  const int64_t end =
      base + (int64_t)block_inclusive_scan_u64((uint64_t)mine.need, scratch, &total);
  const bool granted = mine.valid && (mine.need == 0 || end <= n_free);
  if (tid < n) {
    s_off[tid] = granted ? end - mine.need : -1;
    s_held[tid] = mine.held;
    s_need[tid] = mine.need;
    s_bad[tid] = 0u;
  }
  // the blocks granted: the largest sum not above the list's length.  The sums
  // never fall, so one CTA sees that length inside its range, or the last one
  // ends below it.
  const int64_t cta_end = base + (int64_t)total;
  const bool last = first + n == p.B;
  if (blockIdx.y == 0 && base <= n_free && (cta_end > n_free || last)) {
    const uint64_t under = (tid < n && end <= n_free) ? (uint64_t)end : (uint64_t)base;
    const uint64_t most = block_reduce(under, OpMaxU64(), scratch);
    if (tid == 0) p.taken[0] = (int32_t)most;
  }
  __syncthreads();

  // a parent of a live node must come before it
  if (p.parents) {
    for (int i = tid; i < n * p.max_new; i += kPlanThreads) {
      const int r = i / p.max_new, t = i - r * p.max_new;
      const int parent = p.parents[(int64_t)first * p.max_new + i];
      if (DSPARK_CHECK(i < kPlanCells)) s_parent[i] = parent;
      if (s_off[r] >= 0 && t < p.added[first + r] && (parent >= t || parent < -1)) s_bad[r] = 1u;
    }
    __syncthreads();
  }

  if (blockIdx.y == 0) {
    if (tid < n)
      p.status[first + tid] = !mine.valid    ? DSPARK_ST_BAD_LENGTH
                              : !granted     ? DSPARK_ST_NO_BLOCKS
                              : s_bad[tid]   ? DSPARK_ST_BAD_TREE
                                             : DSPARK_ST_OK;
    // the granted blocks enter the table, a warp per request
    for (int r = tid >> 5; r < n; r += kPlanThreads / 32) {
      const int64_t off = s_off[r];
      if (off < 0) continue;
      int32_t* row = p.table + (int64_t)(first + r) * p.table_ld + s_held[r];
      for (int i = tid & 31; i < s_need[r]; i += 32)
        if (DSPARK_CHECK(off + i < p.max_free && s_held[r] + i < p.max_blocks))
          row[i] = p.free_blocks[off + i];
    }
  }

  // slots, positions and masks
  const int t0 = blockIdx.y * p.span, span = min(p.span, p.max_new - t0);
  for (int i = tid; i < n * span; i += kPlanThreads) {
    const int r = i / span, t = t0 + (i - r * span);
    const int b = first + r;
    const int64_t cell = (int64_t)b * p.max_new + t;
    const int64_t off = s_off[r];
    int slot = -1, position = -1;
    uint64_t mask = 0;
    if (off >= 0 && t < p.added[b]) {
      const int pos = p.ctx[b] + t;  // below max_blocks * page for a valid request
      const int at = pos / p.page;
      const int block = at < s_held[r] ? p.table[(int64_t)b * p.table_ld + at]
                                       : p.free_blocks[off + at - s_held[r]];
      const int64_t s = (int64_t)block * p.page + (pos - at * p.page);
      if (block >= 0 && s <= INT32_MAX) slot = (int)s;
      if (!p.parents) {
        position = pos;
        mask = t < 64 ? ~0ull >> (63 - t) : 0ull;
      } else if (!s_bad[r]) {
        int depth = -1;
        for (int j = t; j >= 0; j = s_parent[r * p.max_new + j]) {  // strictly falling: ends
          mask |= 1ull << j;
          ++depth;
        }
        position = p.ctx[b] + depth;
      }
    }
    p.slots[cell] = slot;
    if (p.positions) p.positions[cell] = position;
    if (p.mask) p.mask[cell] = mask;
  }
}

cudaError_t launch_cache_plan(const int32_t* ctx, const int32_t* added, int B, int max_new,
                              int page, int32_t* table, int64_t table_ld, int max_blocks,
                              const int32_t* free_blocks, int max_free, const int32_t* n_free,
                              const int32_t* parents, int32_t* slots, int32_t* positions,
                              uint64_t* mask, int32_t* taken, int32_t* status,
                              cudaStream_t stream) {
  PlanParams p;
  p.ctx = ctx;
  p.added = added;
  p.B = B;
  p.max_new = max_new;
  p.page = page;
  p.table = table;
  p.table_ld = table_ld;
  p.max_blocks = max_blocks;
  p.free_blocks = free_blocks;
  p.max_free = max_free;
  p.n_free = n_free;
  p.parents = parents;
  p.slots = slots;
  p.positions = positions;
  p.mask = mask;
  p.taken = taken;
  p.status = status;
  // one pair a thread while that makes no more CTAs than the GPU holds at
  // once, else four: a CTA's time is its chain of loads, not its pairs
  const int cells = (int64_t)B * max_new <= 1024 * kPlanThreads ? kPlanThreads : kPlanCells;
  p.group = max_new >= cells ? 1 : cells / max_new;
  if (p.group > kPlanMaxGroup) p.group = kPlanMaxGroup;
  p.span = max_new < cells ? max_new : cells;
  const dim3 grid((B + p.group - 1) / p.group, (max_new + p.span - 1) / p.span);
  cache_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------ cache write
// A piece is 8 elements of one token and head: 16 bytes written; 16 read, or
// 32 from fp32.  2^lane_bits lanes take one token, its keys and its values,
// so that the token's slot is worked out once for all its pieces, and each
// keeps kUnroll pieces of both in flight.  Bound by HBM: 65,536 tokens of 8
// heads of 128 from fp32 take 119 us, 6.8 TB/s.  (A thread per piece, with the
// slot's divisions in each: 270 us.)
namespace {

constexpr int kWriteThreads = 256;

struct WriteParams {
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  int64_t src_token, src_head;              // elements
  int64_t block_stride, token_stride, head_stride;
  int n_src, n_tokens;
  int vecs, per;                            // pieces of a head's row, of a token
  int n_blocks, page, lane_bits;
  const int32_t* slots;
  const int32_t* rows;
};

template <typename T>
__device__ __forceinline__ uint32_t round_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t round_pair<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t round_pair<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

// one piece as it is stored
template <typename T>
__device__ __forceinline__ uint4 stored(const float4 (&f)[2]) {
  return make_uint4(round_pair<T>(f[0].x, f[0].y), round_pair<T>(f[0].z, f[0].w),
                    round_pair<T>(f[1].x, f[1].y), round_pair<T>(f[1].z, f[1].w));
}
template <typename T>
__device__ __forceinline__ uint4 stored(const uint4 (&w)[1]) {
  return w[0];
}

template <typename T, bool kFromF32>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const WriteParams p) {
  using Src = std::conditional_t<kFromF32, float, T>;
  using Load = std::conditional_t<kFromF32, float4, uint4>;
  constexpr int kLoads = kFromF32 ? 2 : 1;
  constexpr int kUnroll = kFromF32 ? 2 : 4;
  const int lanes = 1 << p.lane_bits;
  const int64_t thread = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x;
  const int64_t token = thread >> p.lane_bits;
  if (token >= p.n_tokens) return;
  const int slot = p.slots[token];
  const int64_t row = p.rows ? p.rows[token] : token;
  if (slot < 0 || slot >= p.n_blocks * p.page || row < 0 || row >= p.n_src) return;
  const int block = slot / p.page;
  const int64_t to = block * p.block_stride + (int64_t)(slot - block * p.page) * p.token_stride;
  const Src* k = static_cast<const Src*>(p.k) + row * p.src_token;
  const Src* v = static_cast<const Src*>(p.v) + row * p.src_token;
  for (int j0 = (int)threadIdx.x & (lanes - 1); j0 < p.per; j0 += kUnroll * lanes) {
    Load a[kUnroll][kLoads], c[kUnroll][kLoads];
    int64_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * lanes;
      if (j >= p.per) continue;
      const int head = j / p.vecs, d = (j - head * p.vecs) * 8;
      if (!DSPARK_CHECK(block < p.n_blocks && slot - block * p.page < p.page &&
                        (head + 1) * p.vecs <= p.per && d / 8 < p.vecs && row < p.n_src)) {
        at[u] = -1;
        continue;
      }
      const int64_t from = head * p.src_head + d;
      at[u] = to + head * p.head_stride + d;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        a[u][i] = __ldcs(reinterpret_cast<const Load*>(k + from) + i);
        c[u][i] = __ldcs(reinterpret_cast<const Load*>(v + from) + i);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (j0 + u * lanes >= p.per || !DSPARK_CHECK(at[u] >= 0)) continue;
      *reinterpret_cast<uint4*>(static_cast<T*>(p.k_cache) + at[u]) = stored<T>(a[u]);
      *reinterpret_cast<uint4*>(static_cast<T*>(p.v_cache) + at[u]) = stored<T>(c[u]);
    }
  }
}

cudaError_t launch_kv_write(const void* k, const void* v, int src_dtype, int64_t src_token,
                            int64_t src_head, int n_src, int n_heads, int head_dim, void* k_cache,
                            void* v_cache, int cache_dtype, int64_t block_stride,
                            int64_t token_stride, int64_t head_stride, int n_blocks, int page,
                            const int32_t* slots, const int32_t* rows, int n_tokens,
                            cudaStream_t stream) {
  WriteParams p;
  p.k = k;
  p.v = v;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.src_token = src_token;
  p.src_head = src_head;
  p.block_stride = block_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.n_src = n_src;
  p.n_tokens = n_tokens;
  p.vecs = head_dim / 8;
  p.per = n_heads * p.vecs;
  p.n_blocks = n_blocks;
  p.page = page;
  p.slots = slots;
  p.rows = rows;
  p.lane_bits = 0;  // as many lanes as the token has pieces, at most a warp
  while (p.lane_bits < 5 && (2 << p.lane_bits) <= p.per) ++p.lane_bits;
  const int64_t threads = (int64_t)n_tokens << p.lane_bits;
  const unsigned grid = (unsigned)((threads + kWriteThreads - 1) / kWriteThreads);
  const bool wide = src_dtype == DSPARK_F32;
  using B16 = __nv_bfloat16;
  if (cache_dtype == DSPARK_BF16 && wide)
    kv_write_kernel<B16, true><<<grid, kWriteThreads, 0, stream>>>(p);
  else if (cache_dtype == DSPARK_BF16)
    kv_write_kernel<B16, false><<<grid, kWriteThreads, 0, stream>>>(p);
  else if (wide)
    kv_write_kernel<__half, true><<<grid, kWriteThreads, 0, stream>>>(p);
  else
    kv_write_kernel<__half, false><<<grid, kWriteThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

DSPARK_CHECK_COLLECTOR(cache)

}  // namespace dspark
