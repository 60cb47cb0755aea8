// tree_attention.cuh -- the kernels of dspark_tree_attention, shared by the
// translation units that instantiate them (one per head_dim).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {
namespace attn {

struct Params {
  const void* q;
  int64_t q_req, q_node, q_head;  // elements, as all strides
  int B, nodes, heads, kv_heads, group;  // group: query heads per cached head
  const void* k;
  const void* v;
  int64_t block_stride, token_stride, head_stride;
  int n_blocks, page;
  const int32_t* table;
  int64_t table_ld;
  int max_blocks;
  const int32_t* ctx;
  const int32_t* n_nodes;
  const uint64_t* mask;
  float scale2;  // scale * log2(e): scores are kept in units of log2
  void* out;
  float* lse;
  int32_t* status;
  char* workspace;
  int max_ctas;   // ranges that the workspace has room for
  int tile;       // positions of a tile
  int item_cost;  // an item's start and end, in tiles
  int row_tiles;  // tiles of an item's rows: ceil(nodes * group / rows per CTA)
  int part_rows;  // rows of a partial result in the workspace
  int part_wide;  // elements of a row that lie together there, a power of two
  bool waits;     // the kernel's waits can expire: each CTA writes its Lost
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// the 8 x 8 matrix of 16-bit elements that a warp holds, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The 16-bit types.  The softmax weights are rounded to the inputs' type for
// the second product: the tensor instructions take both operands in one type,
// and a second product for what the rounding leaves over would cost as much
// as the first.  A weight is off by half a step, u of it (2^-8 bf16, 2^-11
// f16), so a result by at most u sum p|v|, as much as by its own rounding
// (against 64 bits 1.2 to 1.35 times the error of fp32 weights, bf16 2.1e-3
// relative).  The sum is taken before the rounding, as lse would be off by u
// after it.
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static constexpr uint32_t kExponent = 0x7F80u;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float widen(uint32_t h) { return __uint_as_float(h << 16); }
};
template <>
struct Half<__half> {
  static constexpr uint32_t kExponent = 0x7C00u;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float widen(uint32_t h) {
    return __half2float(__ushort_as_half((unsigned short)h));
  }
};

// whether either 16-bit half is an infinity or a NaN
template <typename T>
__device__ __forceinline__ bool any_special(uint32_t w) {
  constexpr uint32_t e = Half<T>::kExponent;
  return (w & e) == e || ((w >> 16) & e) == e;
}
// the halves that are neither; 0 in place of the others
template <typename T>
__device__ __forceinline__ uint32_t without_special(uint32_t w) {
  constexpr uint32_t e = Half<T>::kExponent;
  if ((w & e) == e) w &= 0xFFFF0000u;
  if (((w >> 16) & e) == e) w &= 0x0000FFFFu;
  return w;
}

// --------------------------------------------------------- division of work
// Positions are taken in tiles.  The tiles of all (request, cached head)
// items in a row form one axis, cut into equal ranges, one per team of CTAs,
// so that every SM reads the same number of bytes whatever the lengths.  The
// CTAs of a team take one tile of the item's rows each and go over the same
// keys at the same time, so that all but the first find them in L2.  An item
// that lies inside one range is finished by its team; the others leave
// partial rows in the workspace for the joining kernel.  Each item has at
// least one tile (a request without tokens still writes its zero rows), and
// counts for item_cost tiles more, ahead of its first: the time that its
// queries, its first copies and its results take, without which the teams
// that get many short items end last.  (A pair of ranges in one CTA counts as
// two CTAs here.)  The costs by kernel, from what an item takes beside its
// tiles, and requests of mixed lengths at 0, about half, the value and double
// of it (us): streaming, 64 requests of 300 to 8,000 tokens and 4 rows, 113,
// 103, 107, 113 (of 300 tokens 66, 66, 67, 68); kPair, the same with 24 rows,
// 115, 112, 113, 114; kBoth, 64 of 30 to 1,000 tokens and 512 rows, 138, 95,
// 89, 100 (head_dim 64: 98, 69, 74, 84); kOne, 64 of 300 to 8,000 tokens, 219
// at 0, 210 at 1, 204 at 2, 206 at 4.  The streaming and kOne values are not
// their best.
// A range is at least kMinRange long: the join of more parts costs more than they save.
constexpr int kMinRange = 3;
constexpr int kStreamCost = 5, kPairCost = 2, kBothCost = 8, kOneCost = 1;

struct Start {  // where a team's range begins: `at` into the item, of item_cost + tiles
  int b, head, at, tiles;
};

// The item that is cut first at a team's start, after the team before began
// it: what the joining kernel has to join there, up to team `last` (-1: the
// start lies between items, or the item was cut before).
struct Seam {
  int b, head, last, none;
};

// The requests of a CTA's range when one of its waits expired (none: first > last).  Their
// status is written by the joining kernel, after every CTA that may have called them well.
struct Lost {
  int first, last;
};

struct Workspace {
  Seam* seam;     // [ctas], by team
  Lost* lost;     // [ctas]
  float2* stats;  // [2 * ctas][rows]: the reference of the exponents, the sum
  float* rows;    // [2 * ctas][dim / wide][rows][wide]
};

__host__ __device__ inline int64_t workspace_bytes(int rows, int dim, int ctas) {
  return 32 + (int64_t)ctas * (sizeof(Seam) + sizeof(Lost)) +
         2ll * ctas * rows * (sizeof(float2) + (int64_t)dim * sizeof(float));
}

__device__ __forceinline__ Workspace carve(char* w, int rows, int ctas) {
  Workspace s;  // every part 32-byte aligned
  w = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(w) + 31) & ~(uintptr_t)31);
  s.seam = reinterpret_cast<Seam*>(w);
  s.lost = reinterpret_cast<Lost*>(w + ctas * sizeof(Seam));
  s.stats = reinterpret_cast<float2*>(w + ctas * (sizeof(Seam) + sizeof(Lost)));
  s.rows = reinterpret_cast<float*>(s.stats + 2 * ctas * rows);
  return s;
}

// Element d of partial row r of the result whose first row is `slot`.  A row
// lies in one piece where lanes write along it; in pieces of 8 (32 bytes)
// where a warp has a row a lane and many rows, so that it writes whole lines
// (wide trees 148 -> 146 us; elsewhere the joins' reads lose 1 %).
__device__ __forceinline__ float* part_at(const Workspace& ws, int64_t slot, int rows, int wide,
                                          int r, int dim, int d) {
  return ws.rows + slot * dim + ((int64_t)(d / wide) * rows + r) * wide + d % wide;
}

// Bounds of the checked build: row r of the partial result at `slot`, and a row of out and lse.
__device__ __forceinline__ bool part_held(const Params& p, int64_t slot, int r) {
  return r >= 0 && r < p.part_rows && slot >= 0 && slot % p.part_rows == 0 &&
         slot < 2ll * p.max_ctas * p.part_rows;
}
__device__ __forceinline__ bool row_held(const Params& p, int64_t to) {
  return to >= 0 && to < (int64_t)p.B * p.nodes * p.heads;
}

// a request's tokens: the cached text, and all with its nodes (0 when refused)
struct Lengths {
  int ctx, len, nodes;
  bool bad;
};

__device__ __forceinline__ Lengths request_lengths(const Params& p, int b) {
  Lengths r;
  r.ctx = p.ctx[b];
  r.nodes = p.n_nodes[b];
  r.bad = r.ctx < 0 || r.nodes < 0 || r.nodes > p.nodes ||
          (int64_t)r.ctx + r.nodes > (int64_t)p.max_blocks * p.page;
  if (r.bad) r.ctx = r.nodes = 0;
  r.len = r.nodes > 0 ? r.ctx + r.nodes : 0;  // no row: nothing to read
  return r;
}

// an item's tiles of `tile` positions
__device__ __forceinline__ int tiles_of(const Lengths& r, int tile) {
  return r.len > 0 ? (r.len - 1) / tile + 1 : 1;
}

// 64 bits by 32: in 32 bits where that is enough, as it nearly always is
__device__ __forceinline__ int64_t divide(int64_t a, int32_t b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The axis cut into ranges that differ by one at most: the first `more` of
// them have one point more than the others.
struct Cut {
  int64_t per;
  int teams, more;
  // the first point of team c's range, and the team whose range holds point x
  __device__ __forceinline__ int64_t first_of(int c) const { return c * per + min(c, more); }
  __device__ __forceinline__ int owner_of(int64_t x) const {
    const int64_t head = more * (per + 1);
    if (x < head) return (int)(per >= INT32_MAX ? x / (per + 1) : divide(x, (int)per + 1));
    return more + (int)(per >= INT32_MAX ? (x - head) / per : divide(x - head, (int)per));
  }
};
__device__ __forceinline__ Cut cut(int64_t total, int teams) {
  Cut c;
  c.teams = (int)max(1ll, min((long long)teams, (long long)total / kMinRange));
  c.per = divide(total, c.teams);
  c.more = (int)(total - c.per * c.teams);
  return c;
}

// This thread's part [before, upto) of the axis, that of its share of the
// requests; returns the axis' length.  All threads of the block call.
template <int kBlock>
__device__ __forceinline__ int64_t axis_part(const Params& p, uint64_t* scan, int64_t* before,
                                             int64_t* upto) {
  const int per = (p.B + kBlock - 1) / kBlock;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  uint64_t sum = 0, total;
  for (int b = b0; b < b1; ++b)
    sum += (uint64_t)(tiles_of(request_lengths(p, b), p.tile) + p.item_cost) * p.kv_heads;
  *upto = (int64_t)block_inclusive_scan_u64(sum, scan, &total);
  *before = *upto - (int64_t)sum;
  return (int64_t)total;
}
// where point x of the axis lies, if it is in this thread's part
template <int kBlock>
__device__ __forceinline__ bool locate(const Params& p, int64_t before, int64_t upto, int64_t x,
                                       Start* start) {
  if (x < before || x >= upto) return false;
  for (int b = (int)threadIdx.x * ((p.B + kBlock - 1) / kBlock);; ++b) {  // ends by x < upto
    const int tiles = tiles_of(request_lengths(p, b), p.tile);
    const int item = tiles + p.item_cost;
    const int64_t end = before + (int64_t)item * p.kv_heads;
    if (x < end) {
      const int head = (int)divide(x - before, item);
      *start = {b, head, (int)(x - before - (int64_t)head * item), tiles};
      return true;
    }
    before = end;
  }
}

// A CTA's way along its range, item by item.
struct Walk {
  int64_t left;       // of the range
  int b, head, tiles;
  int at;             // into the item
  int cost;           // an item's, ahead of its tiles
  int first, count;   // the tiles of the item that are this CTA's
  Lengths len;        // of request b
  // on to the next item of which a tile is this CTA's; false at the end
  __device__ __forceinline__ bool advance(const Params& p, int tile) {
    count = 0;
    while (left > 0 && count == 0) {
      if (at < 0) {  // the item before is done
        at = 0;
        if (++head == p.kv_heads) {
          head = 0;
          len = request_lengths(p, ++b);
          tiles = tiles_of(len, tile);
        }
      }
      const int take = (int)min(left, (int64_t)(cost + tiles - at));
      first = max(0, at - cost);
      count = max(0, at + take - cost) - first;
      left -= take;
      at = -1;
    }
    return count > 0;
  }
  __device__ __forceinline__ bool whole() const { return count == tiles; }
  __device__ __forceinline__ int64_t slot(int cta) const {  // of the partial rows
    return 2ll * cta + (first == 0 ? 1 : 0);
  }
};
__device__ __forceinline__ Walk walk_from(const Params& p, const Start& s, int64_t left,
                                           int cost) {
  Walk w;
  w.left = left;
  w.cost = cost;
  w.b = s.b;
  w.head = s.head;
  w.tiles = s.tiles;
  w.at = s.at;
  w.first = w.count = 0;
  w.len = {0, 0, 0, false};
  if (left > 0) w.len = request_lengths(p, s.b);
  return w;
}

// This CTA's ranges of the tile axis, kStreams of them side by side: their
// lengths (0: no work), and where they begin (shared memory, valid after the
// call).  All threads call.
template <int kBlock, int kStreams>
__device__ __forceinline__ void find_range(const Params& p, const Workspace& ws, uint64_t* scan,
                                           Start* start, int64_t* range) {
  int64_t before, upto;
  const int64_t total = axis_part<kBlock>(p, scan, &before, &upto);
  const Cut c = cut(total, gridDim.x * kStreams / p.row_tiles);
#pragma unroll
  for (int x = 0; x < kStreams; ++x) {
    const int team = blockIdx.x / p.row_tiles * kStreams + x;
    range[x] = 0;
    if (team >= c.teams) continue;
    const int64_t x0 = c.first_of(team);
    range[x] = c.first_of(team + 1) - x0;
    if (locate<kBlock>(p, before, upto, x0, &start[x]) && blockIdx.x % p.row_tiles == 0) {
      const Start at = start[x];
      Seam seam = {at.b, at.head, -1, 0};
      const int64_t begin = x0 - at.at + p.item_cost;  // the item's first tile
      if (at.at > p.item_cost && c.owner_of(begin) == team - 1)
        seam.last = c.owner_of(begin + at.tiles - 1);
      if (DSPARK_CHECK(team < p.max_ctas && at.b < p.B && at.head < p.kv_heads &&
                       seam.last < c.teams))
        ws.seam[team] = seam;
    }
  }
  // teams without work: nothing to join
  for (int t = c.teams + blockIdx.x * kBlock + threadIdx.x;
       t < (int)gridDim.x * kStreams / p.row_tiles; t += gridDim.x * kBlock)
    if (DSPARK_CHECK(t < p.max_ctas)) ws.seam[t] = {0, 0, -1, 0};
  __syncthreads();
}

// ------------------------------------------------------ the streaming kernel
// For up to 64 rows of an item.  A row is one query head of one node; all
// rows of an item read the same keys, so they stand side by side.
//
// Products: the transposed forms S^T = K Q^T and O^T = V^T P^T on m16n8k16
// (16 keys or 16 dims by 8 rows), so the rows are padded to eights only, K
// and V are the first operand straight from shared memory (ldmatrix; V
// through its transposing form), Q stays in registers as the second, and the
// weights go from the accumulators of S^T to the second operand of the next
// product by one 8 x 8 transpose in registers.
//
// Softmax: each row keeps a reference r (of which the exponents are taken
// off), a sum and the accumulators.  A step whose scores all stay below
// r + 8 leaves r alone, so most steps need no maximum across the warp and no
// rescaling: the weights stay below 2^8 and the sums far inside fp32.
//
// Warps: KW groups of MW warps.  A group takes every KW-th step of 16 keys,
// with its own ring of asynchronous copies and its own softmax state: no
// barrier in the loop but the pair's own.  The MW warps of a group share its
// keys and split the rows.  Groups are joined in shared memory at the end of
// an item.
//
// Bound by HBM: 16 steps of 8 KB are in flight per SM at head_dim 128.  256
// items of 4,000 tokens and 8 rows take 90 us (5.8 TB/s), two requests of
// 100,000 tokens 133 us (6.1 TB/s).
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 16;
constexpr float kSlack = 8.0f;

template <int D, int N8, int MW>
struct Shape {
  static constexpr int kGroups = kWarps / MW;
  static constexpr int kTile = kKeys * kGroups;       // positions a CTA takes at once
  static constexpr int kRows = 8 * N8 * MW;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;
  static constexpr int kCtas = D == 256 ? 1 : D == 64 && N8 <= 2 ? 4 : 2;  // per SM
  static constexpr int kSmem = 196608 / kCtas;
  static constexpr int kStages = kSmem / (kGroups * kStageBytes);
  static constexpr int kPitch = D + 4;                // floats of a joined row: no bank twice
  static_assert(kGroups * kRows * kPitch * 4 <= kSmem, "the joined rows fit the copies' memory");
};

template <typename T, int D, int N8, int MW>
__global__ void __launch_bounds__(kThreads, Shape<D, N8, MW>::kCtas)
    tree_attention_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, N8, MW>;
  using H = Half<T>;
  constexpr int KW = S::kGroups, kStages = S::kStages, kRows = S::kRows;
  constexpr int kChunks = D / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_scan[32];
  __shared__ Start s_start;
  __shared__ uint32_t s_valid[KW][kStages];
  __shared__ float2 s_stat[KW][kRows];
  __shared__ float s_factor[KW][kRows];  // of each group's part of a row
  __shared__ float2 s_joined[kRows];     // the row's reference and sum
  __shared__ uint64_t s_mask[kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mw = warp % MW, kw = warp / MW;
  const Workspace ws = carve(p.workspace, p.part_rows, p.max_ctas);
  int64_t range;
  find_range<kThreads, 1>(p, ws, s_scan, &s_start, &range);
  Walk cur = walk_from(p, s_start, range, p.item_cost);
  const int r0 = (blockIdx.x % p.row_tiles) * kRows;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const T* kc = static_cast<const T*>(p.k);
  const T* vc = static_cast<const T*>(p.v);
  const bool whole = p.page % kKeys == 0;  // a step lies in one block
  const uint32_t ring = smem_u32(smem) + kw * kStages * S::kStageBytes;

  while (cur.advance(p, S::kTile)) {
    const int tiles = cur.count;
    const Lengths len = cur.len;
    const int kvh = cur.head;
    const int32_t* table = p.table + cur.b * p.table_ld;
    const int live = len.nodes * p.group;  // rows below this one have a node

    if (tid == 0 && r0 == 0 && kvh == 0 && cur.first == 0)
      p.status[cur.b] = len.bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;

    // ---- copies: 16 positions of this group into a stage of its ring
    const int first = cur.first * S::kTile + kw * kKeys;  // this group's first position
    const int64_t head_off = kvh * p.head_stride;
    auto entry_of = [&](int step) -> int {  // the block of this lane's position in a step
      const int pos = first + step * S::kTile + (whole ? 0 : (lane & 15));
      return step < tiles && pos < len.len &&
                     DSPARK_CHECK(pos >= 0 && pos / p.page < p.max_blocks && cur.b < p.B)
                 ? __ldg(table + pos / p.page)
                 : -1;
    };
    auto issue = [&](int step, int block) {
      const int pos = first + step * S::kTile;
      const int mine = pos + (whole ? 0 : (lane & 15));
      const bool held = block >= 0 && block < p.n_blocks && mine < len.len;
      const int64_t off = held ? block * p.block_stride +
                                     (int64_t)(mine - mine / p.page * p.page) * p.token_stride
                               : 0;
      uint32_t valid = __ballot_sync(0xffffffffu, held) & 0xFFFFu;
      if (whole) valid = held ? (len.len - pos >= 16 ? 0xFFFFu : (1u << (len.len - pos)) - 1u) : 0u;
      const int stage = step % kStages;
      if (lane == 0 && mw == 0) s_valid[kw][stage] = valid;
      const uint32_t to = ring + stage * S::kStageBytes;
#pragma unroll
      for (int i = 0; i < kKeys * kChunks / (32 * MW); ++i) {
        const int at = (i * MW + mw) * 32 + lane;
        const int row = at / kChunks, chunk = at % kChunks;
        // a step of whole blocks lies in one of them
        const bool on = ((valid >> row) & 1u) &&
                        DSPARK_CHECK(kvh < p.kv_heads && pos + row < len.len &&
                                     (!whole || pos % p.page + row < p.page));
        const int64_t row_off = whole ? off + row * p.token_stride
                                      : __shfl_sync(0xffffffffu, (long long)off, row);
        const int64_t from = on ? row_off + head_off + chunk * 8 : 0;
        const uint32_t d = to + row * S::kRowBytes + ((chunk ^ (row & 7)) << 4);
        cp_async16(d, kc + from, on);
        cp_async16(d + kKeys * S::kRowBytes, vc + from, on);
      }
    };
    int ahead = entry_of(0);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      const int block = ahead;
      ahead = entry_of(s + 1);
      if (s < tiles) issue(s, block);
      cp_async_commit();
    }

    // ---- the rows: masks, and Q as the second operand's fragments
    for (int r = tid; r < kRows; r += kThreads) {
      const int row = r0 + r, node = row / p.group;
      uint64_t m = 0;
      if (row < live && DSPARK_CHECK(node < p.nodes && cur.b < p.B)) {
        m = p.mask ? p.mask[(int64_t)cur.b * p.nodes + node] : ~0ull >> (63 - node);
      }
      s_mask[r] = m;
    }
    uint32_t q[D / 16][N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n) {
      const int row = r0 + (mw * N8 + n) * 8 + (lane >> 2);
      const int node = row / p.group, h = kvh * p.group + row - node * p.group;
      const T* from = static_cast<const T*>(p.q) + cur.b * p.q_req + node * p.q_node +
                      h * p.q_head + (lane & 3) * 2;
      const bool has = row < live && DSPARK_CHECK(cur.b < p.B && node < p.nodes && h < p.heads);
#pragma unroll
      for (int kt = 0; kt < D / 16; ++kt) {
        q[kt][n][0] = has ? __ldg(reinterpret_cast<const uint32_t*>(from + kt * 16)) : 0u;
        q[kt][n][1] = has ? __ldg(reinterpret_cast<const uint32_t*>(from + kt * 16 + 8)) : 0u;
      }
    }
    float o[D / 16][N8][4];
    float ref[N8][2], l[N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n) {
      ref[n][0] = ref[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.0f;
    }
    __syncthreads();

    for (int step = 0; step < tiles; ++step) {
      cp_async_wait<kStages - 2>();
      if constexpr (MW == 1)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + kw), "n"(32 * MW) : "memory");
      if (step + kStages - 1 < tiles) {
        const int block = ahead;
        ahead = entry_of(step + kStages);
        issue(step + kStages - 1, block);
      }
      cp_async_commit();
      const int stage = step % kStages;
      const uint32_t valid = s_valid[kw][stage];
      if (valid == 0u) continue;
      const uint32_t kbase = ring + stage * S::kStageBytes;
      const uint32_t vbase = kbase + kKeys * S::kRowBytes;
      const int pos = first + step * S::kTile;

      float s[N8][4];
#pragma unroll
      for (int n = 0; n < N8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
      const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int kt = 0; kt < D / 16; ++kt) {
        uint32_t a[4];
        const int chunk = 2 * kt + (lane >> 4);
        ldmatrix4(a, kbase + krow * S::kRowBytes + ((chunk ^ (krow & 7)) << 4));
#pragma unroll
        for (int n = 0; n < N8; ++n) H::mma(s[n], a, q[kt][n][0], q[kt][n][1]);
      }

      // element e of s[n]: key lane / 4 + 8 (e / 2), row 8 n + 2 (lane % 4) + e % 2
      const bool nodes_here = pos + kKeys > len.ctx;
      bool special = false;
      if (nodes_here || valid != 0xFFFFu) {
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = (lane >> 2) + (e >> 1) * 8;
            bool on = (valid >> key) & 1u;
            const int node = pos + key - len.ctx;
            if (on && node >= 0)
              on = (s_mask[(mw * N8 + n) * 8 + (lane & 3) * 2 + (e & 1)] >> node) & 1ull;
            s[n][e] = on ? s[n][e] * p.scale2 : -INFINITY;
          }
        if (nodes_here) {  // values that some rows see and others do not: any not finite?
          for (int i = lane; i < kKeys * kChunks; i += 32) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(vbase + i * 16));
            special |= any_special<T>(w[0]) || any_special<T>(w[1]) || any_special<T>(w[2]) ||
                       any_special<T>(w[3]);
          }
          special = __any_sync(0xffffffffu, special);
        }
      } else {
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= p.scale2;
      }

      bool over = false;
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) over |= s[n][e] > ref[n][e & 1] + kSlack;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[n][e], s[n][e + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top, ref[n][e]);
            const float scale = top == -INFINITY ? 1.0f : exp2_approx(ref[n][e] - top);
            ref[n][e] = top;
            l[n][e] *= scale;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              o[mt][n][e] *= scale;
              o[mt][n][e + 2] *= scale;
            }
          }
      }

      uint32_t w[N8][2];
      float pr[N8][4];
#pragma unroll
      for (int n = 0; n < N8; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float r = ref[n][e & 1];
          pr[n][e] = exp2_approx(s[n][e] - (r == -INFINITY ? 0.0f : r));
          l[n][e & 1] += pr[n][e];
        }
        w[n][0] = transpose8x8(H::pack(pr[n][0], pr[n][1]));
        w[n][1] = transpose8x8(H::pack(pr[n][2], pr[n][3]));
      }

      const int vrow = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        uint32_t a[4];
        const int chunk = 2 * mt + ((lane >> 3) & 1);
        ldmatrix4_trans(a, vbase + vrow * S::kRowBytes + ((chunk ^ (vrow & 7)) << 4));
        if (special) {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = without_special<T>(a[i]);
        }
#pragma unroll
        for (int n = 0; n < N8; ++n) H::mma(o[mt][n], a, w[n][0], w[n][1]);
      }
      if (special) {
        // infinities and NaN, left out above, reach the rows that see their key only
#pragma unroll 1
        for (int key = 0; key < kKeys; ++key) {
          const int from = (key & 7) * 4 + (lane & 3);
#pragma unroll
          for (int n = 0; n < N8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float score = __shfl_sync(0xffffffffu, key < 8 ? s[n][e] : s[n][e + 2], from);
              const float weight =
                  __shfl_sync(0xffffffffu, key < 8 ? pr[n][e] : pr[n][e + 2], from);
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int d = mt * 16 + h * 8 + (lane >> 2);
                  unsigned short bits;
                  asm volatile("ld.shared.u16 %0, [%1];"
                               : "=h"(bits)
                               : "r"(vbase + key * S::kRowBytes +
                                     (((d >> 3) ^ (key & 7)) << 4) + (d & 7) * 2));
                  if ((bits & H::kExponent) == H::kExponent && score != -INFINITY)
                    o[mt][n][e + 2 * h] += weight * H::widen(bits);
                }
            }
        }
      }
    }

    // ---- join the groups
    cp_async_wait<0>();
    __syncthreads();
    float* joined = reinterpret_cast<float*>(smem);  // [KW][kRows][kPitch]
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum_l = l[n][e];
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 4);
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 8);
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 16);
        const int r = (mw * N8 + n) * 8 + (lane & 3) * 2 + e;
        if (lane < 4) s_stat[kw][r] = make_float2(ref[n][e], sum_l);
        float* row = joined + (kw * kRows + r) * S::kPitch + (lane >> 2);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          row[mt * 16] = o[mt][n][e];
          row[mt * 16 + 8] = o[mt][n][e + 2];
        }
      }
    __syncthreads();
    const bool full = cur.whole();
    const int64_t slot = cur.slot(blockIdx.x) * p.part_rows;
    for (int r = tid; r < kRows; r += kThreads) {
      const int row = r0 + r;
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < KW; ++g) top = fmaxf(top, s_stat[g][r].x);
      const float safe = top == -INFINITY ? 0.0f : top;
      float all = 0.0f, f[KW];
#pragma unroll
      for (int g = 0; g < KW; ++g) {
        f[g] = exp2_approx(s_stat[g][r].x - safe);
        all += s_stat[g][r].y * f[g];
      }
      // a row of no node: its zero query saw the text all the same
      const float by = row >= live || all == 0.0f ? 0.0f : full ? 1.0f / all : 1.0f;
#pragma unroll
      for (int g = 0; g < KW; ++g) s_factor[g][r] = f[g] * by;
      s_joined[r] = row >= live ? make_float2(-INFINITY, 0.0f) : make_float2(top, all);
    }
    __syncthreads();
    const int rows_here = min(kRows, p.nodes * p.group - r0);
    for (int i = tid; i < rows_here * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r0 + r < live) {
#pragma unroll
        for (int g = 0; g < KW; ++g) {
          const float f = s_factor[g][r];
          const float4 v =
              *reinterpret_cast<const float4*>(joined + (g * kRows + r) * S::kPitch + d);
          a.x += v.x * f;
          a.y += v.y * f;
          a.z += v.z * f;
          a.w += v.w * f;
        }
      }
      if (full) {
        const int row = r0 + r, node = row / p.group;
        const int64_t to = ((int64_t)cur.b * p.nodes + node) * p.heads + kvh * p.group + row -
                           node * p.group;
        if (!DSPARK_CHECK(row_held(p, to))) continue;
        uint2 w;
        w.x = H::pack(a.x, a.y);
        w.y = H::pack(a.z, a.w);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + to * D + d) = w;
        if (d == 0 && p.lse) {
          const float2 j = s_joined[r];
          p.lse[to] = j.y == 0.0f ? -INFINITY : (j.x + log2f(j.y)) * 0.6931471805599453f;
        }
      } else if (DSPARK_CHECK(part_held(p, slot, r))) {
        *reinterpret_cast<float4*>(part_at(ws, slot, p.part_rows, D, r, D, d)) = a;
        if (d == 0) ws.stats[slot + r] = s_joined[r];
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------- the joining kernel
// CTA (x, y, z): eight rows of row tile z of the item that is first cut
// between teams x and x + 1, if there is one, are joined from the teams'
// partial rows, in the teams' order.  A warp takes a row, and kAhead teams'
// parts of it are in flight together: its time is the latency of reading them
// (6 us of 104 at 256 items of 4,000 tokens on 304 ranges).  CTA (x, 0, 0)
// also gives the requests that team x lost their status.
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    tree_attention_join_kernel(const __grid_constant__ Params p, int rows) {
  using H = Half<T>;
  constexpr int kPer = D / 32, kAhead = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Workspace ws = carve(p.workspace, p.part_rows, p.max_ctas);
  if (!DSPARK_CHECK(gridDim.x <= p.max_ctas)) return;
  const Seam at = ws.seam[min(blockIdx.x + 1, gridDim.x - 1)];
  // read at the start, as its latency would follow the rows', and used at the end
  Lost lost = {0, -1};
  if (p.waits && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < p.row_tiles &&
      DSPARK_CHECK(blockIdx.x * p.row_tiles + threadIdx.x < p.max_ctas))
    lost = ws.lost[blockIdx.x * p.row_tiles + threadIdx.x];
  [&] {
    const int c0 = blockIdx.x, c1 = blockIdx.x + 1 < gridDim.x ? at.last : -1;  // the item's teams
    if (c1 < 0) return;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const int row = blockIdx.z * rows + r;
    if (r >= rows || row >= p.nodes * p.group) return;
    // the first partial row of team c: its first range's in slot 0, its last's in slot 1
    auto part_of = [&](int c) -> int64_t {
      return (2ll * (c * p.row_tiles + blockIdx.z) + (c == c0 ? 1 : 0)) * p.part_rows;
    };

    // part_at, with the width's division as a shift
    const int shift = 31 - __clz(p.part_wide), d0 = lane * kPer;
    const int offset =
        ((((d0 >> shift) * p.part_rows) + r) << shift) + (d0 & (p.part_wide - 1));
    if (!DSPARK_CHECK(c1 < gridDim.x && part_held(p, part_of(c0), r) &&
                      part_held(p, part_of(c1), r) && offset + kPer <= p.part_rows * D))
      return;
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, ws.stats[part_of(c) + r].x);
    top = warp_reduce(top, OpMaxF());
    const float safe = top == -INFINITY ? 0.0f : top;
    float all = 0.0f, a[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d) a[d] = 0.0f;
#pragma unroll kAhead
    for (int c = c0; c <= c1; ++c) {
      const float2 st = ws.stats[part_of(c) + r];
      const float* v = ws.rows + part_of(c) * D + offset;
      float x[kPer];
      if constexpr (kPer == 2) {
        *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(v);
      } else {
#pragma unroll
        for (int d = 0; d < kPer; d += 4)
          *reinterpret_cast<float4*>(x + d) = *reinterpret_cast<const float4*>(v + d);
      }
      const float f = exp2_approx(st.x - safe);
      all += st.y * f;
#pragma unroll
      for (int d = 0; d < kPer; ++d) a[d] += x[d] * f;
    }
    const int node = row / p.group, h = at.head * p.group + row - node * p.group;
    const int64_t to = ((int64_t)at.b * p.nodes + node) * p.heads + h;
    if (!DSPARK_CHECK(row_held(p, to))) return;
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int d = 0; d < kPer; d += 2) w[d / 2] = H::pack(a[d] * inv, a[d + 1] * inv);
    uint32_t* out =
        reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + to * D) + lane * (kPer / 2);
    if constexpr (kPer == 2)
      *out = w[0];
    else if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane == 0 && p.lse)
      p.lse[to] = all == 0.0f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
  }();
  for (int b = lost.first; b <= lost.last; ++b) p.status[b] = DSPARK_ST_TIMEOUT;
}

// ---------------------------------------------------------------- launches
// the joining kernel after a kernel of `grid` ranges; it is launched while
// that one runs and waits on the device for its end
template <typename T, int D>
cudaError_t launch_join(const Params& p, int rows, int grid, cudaStream_t stream) {
  const int teams = grid / p.row_tiles;
  if (teams == 1 && !p.waits) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  const int used = min(rows, p.nodes * p.group);
  cfg.gridDim = dim3(teams, (used + kJoinThreads / 32 - 1) / (kJoinThreads / 32), p.row_tiles);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_attention_join_kernel<T, D>, p, rows);
}

// rows of a streaming CTA for `rows` rows of an item
inline int stream_rows(int rows, int dim) {
  if (dim == 256) return rows <= 8 ? 8 : rows <= 16 ? 16 : 64;
  return rows <= 24 ? (rows + 7) / 8 * 8 : rows <= 32 ? 32 : 64;
}
// Rows up to which the streaming kernel is taken (256 items of 4,000 tokens / 4,096 of 60, us,
// against the tensor kernel).  head_dim 64: 16 rows 55 / 38 against 59 / 50, 24 rows 67 / 81
// against 60 / 73.  128: 8 rows 88 / 62 against 92 / 62, 16 rows 91 / 83 against 93 / 63.  256:
// 1 row 185 / 120 against 163 / 135, 8 rows 187 / 159 against 166 / 142.  These are batches: one
// request alone, of 4,000 tokens with 24 rows at head_dim 64, takes 16.2 streaming and 16.9 in the
// tensor kernel.
constexpr int few_rows(int dim) { return dim == 64 ? 16 : dim == 128 ? 8 : 0; }
// the workspace's ranges, by kernel (160 SMs at most are used), and the rows of
// each: those that the item has, of a CTA's
inline int stream_ctas(int dim, int rows) {
  return 160 * (dim == 256 ? 1 : dim == 64 && rows <= 16 ? 4 : 2);
}
inline int wide_ctas(bool pair) { return pair ? 320 : 160; }
inline int part_rows(int rows, int cta_rows) {
  return rows >= cta_rows ? cta_rows : (rows + 7) / 8 * 8;
}

template <typename T, int D, int N8, int MW>
cudaError_t launch_shape(Params p, int sms, cudaStream_t stream) {
  using S = Shape<D, N8, MW>;
  p.row_tiles = (p.nodes * p.group + S::kRows - 1) / S::kRows;
  auto* kernel = tree_attention_kernel<T, D, N8, MW>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kSmem);
  if (e != cudaSuccess) return e;
  p.part_rows = part_rows(p.nodes * p.group, S::kRows);
  p.part_wide = D;
  p.max_ctas = stream_ctas(D, S::kRows);
  p.item_cost = kStreamCost;
  p.tile = S::kTile;
  p.waits = false;
  const int grid = min(p.max_ctas, max(sms * S::kCtas, p.row_tiles));
  kernel<<<grid, kThreads, S::kSmem, stream>>>(p);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<T, D>(p, S::kRows, grid, stream);
}

cudaError_t launch_64(const Params& p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_128(const Params& p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_256(const Params& p, int dtype, int sms, cudaStream_t stream);

}  // namespace attn
}  // namespace dspark
