// tree_attention_wide.cuh -- the attention kernel on the fifth generation's
// tensor instructions and tensor copies, for caches whose blocks are made of
// groups of eight rows.  Included by the translation units of
// tree_attention.cuh.
#pragma once

#include <cuda.h>

#include "tree_attention.cuh"

// The checked build can leave one CTA of the kernel without its copies, so that its waits expire:
// dspark_debug_stall_attention.
#ifdef DSPARK_CHECKED
static __device__ uint32_t g_stalled;  // the CTA + 1
#define DSPARK_STALLED(cta) (*(volatile uint32_t*)&g_stalled == (cta) + 1u)
#define DSPARK_STALL_SETTER(dim) \
  cudaError_t stall_##dim(uint32_t v) { return cudaMemcpyToSymbol(g_stalled, &v, 4); }
#else
#define DSPARK_STALLED(cta) false
#define DSPARK_STALL_SETTER(dim)
#endif

namespace dspark {
namespace attn {

// ------------------------------------------------- tcgen05 and its barriers
// Shared-memory operand descriptor: start address, leading and stride byte
// offsets (each / 16), version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// One lane of a converged warp: the products' operands are warp-uniform, and
// stay in uniform registers when only the instruction itself is predicated.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0u;
}
// d[tmem] (+)= a b with a and b in shared memory, by the lane with `on`
__device__ __forceinline__ void mma_ss(bool on, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"((uint32_t)on)
      : "memory");
}
// the same with a in tensor memory
__device__ __forceinline__ void mma_ts(bool on, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"((uint32_t)on)
      : "memory");
}
// arrives on `bar` once every product issued before it is done
__device__ __forceinline__ void mma_commit(bool on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// one box of a cache, from row r of block b of head h, dims 64 x .., completing on `bar`; a
// block beyond the cache gives zeros
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, int r, int x,
                                             int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(0), "r"(r), "r"(x), "r"(h), "r"(b), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_load32(float* v, uint32_t addr) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------ the kernel
// S = Q K^T into tensor memory for a tile of 128 rows and 64 positions,
// softmax by the warpgroup that owns the row tile (a thread per row, so no
// exchange between threads), the weights back into tensor memory over the
// scores, O += P V.  The scores of two tiles are held for each row tile, so
// that the products of the next tile run during a softmax, and two warpgroups
// share the tensor cores.  (With tiles of 128 positions, whose scores fill
// the place of two, a row tile's products and softmax wait for one another:
// 1,024 one-row-tile items of 300 tokens 105 us instead of 86, wide trees 165
// instead of 146 at that time; head_dim 64, 2,048 items of 300 tokens 82
// instead of 60.)
//
// kPair: items of up to 128 rows.  The warpgroups go along two ranges of the
//   tile axis, each with its own queries and its own copies of keys and
//   values: two CTAs in one, of which one's starts and results are hidden
//   behind the other's products.  Bound by HBM: 256 items of 4,000 tokens
//   take 95 us with 24 rows, 113 us with 128 (5.6 and 4.8 TB/s), two
//   requests of 131,000 tokens 174 us (6.2 TB/s).
// kBoth: items of more rows.  The warpgroups take two row tiles of one item
//   and share its keys and values.  Bound by the products (2 * 2 * 128 * 64 *
//   D operations a row tile and tile of positions) and by their issue: 256
//   items of 4,000 tokens and 512 rows take 205 us, 1.3 PFLOP/s; 16 requests
//   with trees of 64 nodes and 8 query heads to a cached head 134 to 140 us.  A row
//   tile's twelve products take 640 cycles, as the scores' operands come at
//   the rate of shared memory; the two row tiles' take 1,550 in the loop.
// kOne: head_dim 256, whose accumulators fill half the tensor memory: one
//   warpgroup and one row tile.  256 items of 4,000 tokens take 173 us with
//   24 rows (6.1 TB/s), 466 us with 512, whose four row tiles are four CTAs
//   that copy the same keys, three of them from L2.
//
// A score that passes the row's reference by more than 8 has the accumulators
// rescaled by the softmax warpgroup, once the products before are done; this
// is rare after an item's first tile, as in the streaming kernel.
//
// Warps 0-3 and 4-7: softmax, queries and results.  Warps 8 and 9: tensor
// copies of keys and values, box by box of a block's rows, into a ring of
// stages.  Warps 10 and 11: issue the products of a row tile each.  Q lies in
// rows of 64 dims (128 bytes, swizzled in groups of eight rows), one block of
// 64 dims after the other; keys the same; values too, read with their dims as
// the major axis.
enum WideMode { kPair, kBoth, kOne };

constexpr int kWideThreads = 384;  // 168 registers a thread: a row's 64 scores, 64 of Q, and more

template <int D, WideMode kMode>
struct Wide {
  static constexpr int kStreams = kMode == kPair ? 2 : 1;   // ranges of the tile axis
  static constexpr int kRowTiles = kMode == kOne ? 1 : 2;   // of 128 rows, over all streams
  static constexpr int kRows = kMode == kBoth ? 256 : 128;  // of an item, per CTA
  static constexpr int kKeys = 64;   // positions of a tile
  static constexpr int kScores = 2;  // tiles whose scores are held
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = 128 * D * 2, kTileBytes = kKeys * D * 2;
  static constexpr int kStages = kMode == kBoth || D == 64 ? 4 : 2;
  static constexpr int kPartWide = kMode == kBoth ? 8 : D;  // of a partial row, in one piece
  static constexpr int kRing = 2 * kStages * kTileBytes;    // keys, then values
  static constexpr int kSmem = kRowTiles * kQBytes + kStreams * kRing + 1024;
};
constexpr int kWideMaxStages = 4;

// How a tile comes in boxes of rows of one block.  Keys: boxes of k_rows rows
// of 64 dims, the tile's rows of each 64 dims together; or (k_whole) boxes of
// eight rows of all dims, where those are fewer.  Values: boxes of v_rows rows
// of all dims.
struct Boxes {
  int k_rows, k_whole, v_rows;
};

struct WideStream {
  uint64_t k_full[kWideMaxStages], k_empty[kWideMaxStages];
  uint64_t v_full[kWideMaxStages], v_empty[kWideMaxStages];
  uint32_t valid[8][2];  // a tile's positions that hold a key, by tile number modulo 8
  uint32_t special[8];   // a value of a tile's nodes is an infinity or a NaN
};
struct WideShared {
  WideStream stream[2];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2], turn[2], drained[2];
  uint64_t scan[32];
  int64_t q_row[256];  // where each row of the CTA begins in Q, from its request and cached head on
  Start start[2];
  uint32_t tmem;
  uint32_t failed;  // a wait expired
};

template <typename T, int D, WideMode kMode>
__global__ void __launch_bounds__(kWideThreads, 1)
    tree_attention_wide_kernel(const __grid_constant__ Params p,
                               const __grid_constant__ CUtensorMap k_map,
                               const __grid_constant__ CUtensorMap v_map,
                               const Boxes boxes) {
  using H = Half<T>;
  using W = Wide<D, kMode>;
  constexpr int kChunks = D / 8, kStages = W::kStages, kKeys = W::kKeys, kHalves = W::kHalves;
  constexpr bool kPaired = kMode == kPair;
  extern __shared__ unsigned char smem_raw[];
  __shared__ WideShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + W::kRowTiles * W::kQBytes;
  // bytes between the groups of eight rows of a tile, and between its blocks of 64 dims
  const uint32_t k_group = boxes.k_whole ? kHalves * 1024u : 1024u;
  const uint32_t k_half = boxes.k_whole ? 1024u : kKeys * 128u;
  const uint32_t v_half = boxes.v_rows * 128u, v_box = kHalves * v_half;
  const int v_shift = 31 - __clz(boxes.v_rows);  // a power of two, as k_rows is

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  const Workspace ws = carve(p.workspace, p.part_rows, p.max_ctas);
  int64_t ranges[W::kStreams];
  find_range<kWideThreads, W::kStreams>(p, ws, sh.scan, sh.start, ranges);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < W::kStreams && DSPARK_CHECK(blockIdx.x * W::kStreams + tid < p.max_ctas))
    ws.lost[blockIdx.x * W::kStreams + tid] = {0, -1};
  if (ranges[0] <= 0) return;  // the second stream's range comes behind the first's
  const int r0 = (blockIdx.x % p.row_tiles) * W::kRows;
  // row tiles of one stream
  const int n_tiles = kMode == kBoth && p.nodes * p.group - r0 > 128 ? 2 : 1;

  for (int r = tid; r < W::kRows; r += kWideThreads) {
    const int row = min(r0 + r, p.nodes * p.group - 1), node = row / p.group;  // past the end: the last
    sh.q_row[r] = node * p.q_node + (row - node * p.group) * p.q_head;
  }
  if (tid == 0) {
    for (int x = 0; x < W::kStreams; ++x)
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&sh.stream[x].k_full[i], 1);
        mbar_init(&sh.stream[x].k_empty[i], n_tiles);
        mbar_init(&sh.stream[x].v_full[i], 1);
        mbar_init(&sh.stream[x].v_empty[i], n_tiles);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 128);
      for (int j = 0; j < W::kScores; ++j) {
        mbar_init(&sh.s_full[i][j], 1);
        mbar_init(&sh.p_full[i][j], 128);
      }
      mbar_init(&sh.o_full[i][0], 1);
      mbar_init(&sh.o_full[i][1], 1);
      mbar_init(&sh.turn[i], 32);
      mbar_init(&sh.drained[i], 1);
    }
    sh.failed = 0u;
    mbar_init_fence();
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  // columns: the scores of row tile m and tile g (the weights over their first half), then the
  // accumulators
  const uint32_t tmem = sh.tmem;
  auto s_col = [&](int m, uint32_t g) -> uint32_t {
    return tmem + 128u * m + (g % W::kScores) * 64u;
  };
  auto o_col = [&](int m) -> uint32_t { return tmem + 256u + 128u * m; };

  // A bounded wait of a whole warp; once one expires, every later one of the CTA gives up at once.
  // The lanes poll and leave together: each branch is on a vote of all of them.  So the warp is
  // whole when it goes on to products, whose operands lie in its uniform registers.
  auto wait_all = [&](uint64_t* bar, uint32_t phase) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
    const uint64_t t0 = global_ns();
    uint32_t nap = 32;
    while (!__any_sync(0xffffffffu, *(volatile uint32_t*)&sh.failed)) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
      if (__any_sync(0xffffffffu, global_ns() - t0 >= kWaitLimitNs)) {
        *(volatile uint32_t*)&sh.failed = 1u;
        break;
      }
      if (nap > 32u) __nanosleep(nap);
      nap = nap < 1024u ? 2u * nap : 1024u;
    }
    return false;
  };
  // four waits whose latencies, some 200 cycles each and as long as eight products, overlap; all
  // lanes wait for the same barriers, so the warp stays together
  auto wait_each = [&](uint64_t* const (&bar)[4], const uint32_t (&phase)[4]) -> bool {
    bool done = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) done &= mbar_try_wait(bar[i], phase[i]);
    if (__all_sync(0xffffffffu, done)) return true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!wait_all(bar[i], phase[i])) return false;
    return true;
  };
  auto phase_of = [](uint32_t g) -> uint32_t { return (g / kStages) & 1u; };
  auto score_phase = [](uint32_t g) -> uint32_t { return (g / W::kScores) & 1u; };

  if (warp < 8) {
    // -------------------------------------------------- softmax and results
    const int m = warp >> 2;               // the row tile
    const int x = kPaired ? m : 0;         // the stream
    const int m_rows = r0 + (kPaired ? 0 : m * 128);  // the tile's first row of the item
    WideStream& stream = sh.stream[x];
    const int t = tid & 127;  // this thread's row of the tile and lane of tensor memory
    const uint32_t lanes = (uint32_t)(t & ~31) << 16;
    const uint32_t oc = o_col(m) + lanes;
    const uint32_t q_at = base + m * W::kQBytes;
    // a negative scale goes into Q's sign, so that the largest score stays the largest; 0 would
    // make NaN of a hidden score
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;
    const float scale = fmaxf(fabsf(p.scale2), 1.17549435e-38f);
    uint32_t tile_no = 0;
    bool ok = m < (kPaired ? 2 : n_tiles) && m < W::kRowTiles;
    Walk cur = walk_from(p, sh.start[x], ok ? ranges[x] : 0, p.item_cost);
    // the item's Q: 16-byte pieces of this thread's column, every kStep-th row, in parts of kPart
    constexpr int kStep = 128 / kChunks;
    constexpr int kPart = kChunks > 16 ? 16 : kChunks;
    const int64_t* q_row = sh.q_row + (m_rows - r0) + t / kChunks;
    auto q_from = [&](const Walk& w) -> const T* {
      return static_cast<const T*>(p.q) + w.b * p.q_req + (int64_t)w.head * p.group * p.q_head +
             (t % kChunks) * 8;
    };
    auto prefetch_q = [&](const Walk& w) {  // a thread for each 128-byte line
      if (t % 8 != 0) return;
      const T* from = q_from(w);
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(from + q_row[i * kStep]));
    };
    auto fill_q = [&](const Walk& w) {
      const int live = w.len.nodes * p.group - m_rows, c = t % kChunks;  // rows of the tile
      const T* from = q_from(w);
#pragma unroll
      for (int part = 0; part < kChunks / kPart; ++part) {
        uint4 q[kPart];
        if (!DSPARK_CHECK(w.b < p.B && w.head < p.kv_heads && m_rows - r0 >= 0 &&
                          m_rows - r0 + t / kChunks + (kChunks - 1) * kStep < W::kRows))
          continue;
#pragma unroll
        for (int i = 0; i < kPart; ++i)
          q[i] = __ldg(reinterpret_cast<const uint4*>(from + q_row[(part * kPart + i) * kStep]));
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
          const int r = (part * kPart + i) * kStep + t / kChunks;
          const uint32_t keep = r < live ? ~0u : 0u;
          const uint32_t to = q_at + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          if (!DSPARK_CHECK(to + 16 <= ring)) continue;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to),
                       "r"((q[i].x ^ flip) & keep), "r"((q[i].y ^ flip) & keep),
                       "r"((q[i].z ^ flip) & keep), "r"((q[i].w ^ flip) & keep)
                       : "memory");
        }
      }
      fence_async_shared();
      mbar_arrive(&sh.q_full[m]);
    };
    // tile g's second product is done.  Called for the tile before the one in
    // hand or for an item's last, whose scores say that every product up to
    // two tiles before is: two barriers in turn, so that no phase is mistaken
    // for one two further.
    auto wait_values = [&](uint32_t g) -> bool {
      return wait_all(&sh.o_full[m][g & 1u], (g >> 1) & 1u);
    };
    bool more = ok && cur.advance(p, kKeys);
    if (more) fill_q(cur);
    const int row = m_rows + t, node = row / p.group;
    const bool mine = row < p.nodes * p.group;
    const int64_t my_row = (int64_t)node * p.heads + row - node * p.group;  // in an item's results
    while (ok && more) {
      const int tiles = cur.count;
      const Lengths len = cur.len;
      const int live = len.nodes * p.group;
      if (t == 0 && m_rows == 0 && cur.head == 0 && cur.first == 0)
        p.status[cur.b] = len.bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;

      Walk ahead = cur;
      more = ahead.advance(p, kKeys);
      if (more) prefetch_q(ahead);
      const bool idle = m_rows + (t & ~31) >= live;  // no row of this warp has a node
      uint64_t mask = 0;
      if (row < live && DSPARK_CHECK(node < p.nodes && cur.b < p.B))
        mask = p.mask ? p.mask[(int64_t)cur.b * p.nodes + node] : ~0ull >> (63 - node);
      float ref = -INFINITY;
      float2 sum2 = make_float2(0.0f, 0.0f);
      for (int i = 0; i < tiles; ++i, ++tile_no) {
        ok = wait_all(&sh.s_full[m][tile_no % W::kScores], score_phase(tile_no));
        if (!ok) break;
        tc_after_sync();
        const uint32_t sc = s_col(m, tile_no) + lanes;
        const int pos = (cur.first + i) * kKeys;
        const bool nodes_here = pos + kKeys > len.ctx;
        if (!idle) {
          const uint32_t* words = stream.valid[tile_no & 7u];
          uint32_t all = ~0u;
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) all &= words[c];
          float v[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) tmem_load32(v + c * 32, sc + c * 32);
          tmem_wait_load();
          if (nodes_here || all != ~0u) {
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
              uint32_t w = words[c];
              const int node0 = pos + c * 32 - len.ctx;  // the node of the chunk's first position
              if (node0 >= 0)
                w &= node0 < 64 ? (uint32_t)(mask >> node0) : 0u;
              else if (node0 > -32)
                w &= (uint32_t)(mask << -node0) | ((1u << -node0) - 1u);
              if (__all_sync(0xffffffffu, w == ~0u)) continue;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((w >> j) & 1u)) v[c * 32 + j] = -INFINITY;
            }
          }
          float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int j = 4; j < kKeys - 4; j += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(fmaxf(m4[k], v[j + k]), v[j + 4 + k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], v[kKeys - 4 + k]);
          float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
          if (__any_sync(0xffffffffu, top > ref + kSlack)) {
            top = fmaxf(top, ref);
            const float f = top == -INFINITY ? 1.0f : exp2_approx(ref - top);
            ref = top;
            sum2.x *= f;
            sum2.y *= f;
            if (i > 0) {
              ok = wait_values(tile_no - 1u);
              if (!ok) break;
              tc_after_sync();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t a[16];
                tmem_load16(a, oc + c * 16);
                tmem_wait_load();
#pragma unroll
                for (int j = 0; j < 16; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
                tmem_store16(oc + c * 16, a);
              }
            }
          }
          const float2 off = f2(ref == -INFINITY ? 0.0f : -ref), by = f2(scale);
          float2 part2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < kKeys / 32; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 e = fma2_rn(make_float2(v[c * 32 + 2 * j], v[c * 32 + 2 * j + 1]), by, off);
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              if (j & 1)
                part2 = add2_rn(part2, e);
              else
                sum2 = add2_rn(sum2, e);
              w[j] = H::pack(e.x, e.y);
            }
            tmem_store16(sc + c * 16, w);
          }
          sum2 = add2_rn(sum2, part2);
          tmem_wait_store();
        }
        if (nodes_here && (kMode != kBoth || m == 0)) {
          // Rows from the first node on: nodes, which some rows see and others
          // do not, and what lies behind the end.  0 times an infinity or a
          // NaN would reach rows that do not see it: they are cleared before
          // the weights are handed over, which lets the product begin (of the
          // second row tile after that of the first).
          const uint32_t stage = tile_no % kStages;
          ok = wait_all(&stream.v_full[stage], phase_of(tile_no));
          if (!ok) break;
          const uint32_t v_at = ring + x * W::kRing + (kStages + stage) * W::kTileBytes;
          const int from = max(0, len.ctx - pos);
          // blocks' rows that the last copy brought; zeros behind them
          const int end =
              min(kKeys, (len.len - pos + boxes.v_rows - 1) & -boxes.v_rows);
          const int n = (end - from) * kChunks;
          constexpr int kAtOnce = 4;
          for (int j0 = t; j0 < n; j0 += 128 * kAtOnce) {
            uint32_t addr[kAtOnce], w[kAtOnce][4];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const int j = min(j0 + u * 128, n - 1), r = from + j / kChunks, c = j % kChunks;
              addr[u] = v_at + (r >> v_shift) * v_box + (c >> 3) * v_half +
                        (r & (boxes.v_rows - 1)) * 128 + (((c & 7) ^ (r & 7)) << 4);
              if (!DSPARK_CHECK(addr[u] >= v_at && addr[u] + 16 <= v_at + W::kTileBytes))
                addr[u] = v_at;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                           : "r"(addr[u])
                           : "memory");
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
              if (j0 + u * 128 < n && (any_special<T>(w[u][0]) || any_special<T>(w[u][1]) ||
                                       any_special<T>(w[u][2]) || any_special<T>(w[u][3]))) {
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr[u]),
                             "r"(without_special<T>(w[u][0])), "r"(without_special<T>(w[u][1])),
                             "r"(without_special<T>(w[u][2])), "r"(without_special<T>(w[u][3]))
                             : "memory");
                if (pos + from + (j0 + u * 128) / kChunks < len.len)
                  *(volatile uint32_t*)&stream.special[tile_no & 7u] = 1u;
              }
          }
          __syncwarp();
          fence_async_shared();
        }
        tc_before_sync();
        mbar_arrive(&sh.p_full[m][tile_no % W::kScores]);
      }
      // Q is free, as the last scores are done: the next item's first scores
      // are computed while this one's results are written
      if (ok && more) fill_q(ahead);
      if (ok) ok = wait_values(tile_no - 1u);
      if (!ok) break;
      tc_after_sync();
      // nodes, at most 64, lie in the item's last two tiles (the tiles before these may already
      // have lent their flags to tiles of the next item)
      bool special = false;
      for (uint32_t k = 1; k <= min(2, tiles); ++k)
        special |= stream.special[(tile_no - k) & 7u] != 0u;

      float sum = sum2.x + sum2.y;
      if (row >= live) {  // a row of no node: its zero query saw the text all the same
        ref = -INFINITY;
        sum = 0.0f;
      }
      const bool full = cur.whole();
      const int64_t to = (int64_t)cur.b * p.nodes * p.heads + cur.head * p.group + my_row;
      const int64_t slot = cur.slot(kPaired ? 2 * blockIdx.x + x : blockIdx.x) * p.part_rows;
      const int part_row = (kPaired ? 0 : m * 128) + t;
      const float inv = sum == 0.0f ? 0.0f : full ? 1.0f / sum : 1.0f;
      const int chunks = m_rows + (t & ~31) < p.nodes * p.group ? D / 32 : 0;  // of the warp
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        float v[32];
        tmem_load32(v, oc + c * 32);
        tmem_wait_load();
        if (row >= live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        }
        if (special) {
          // infinities and NaN, left out of the product, reach the rows that see their key
#pragma unroll 1
          for (int k = 0; k < len.nodes; ++k) {
            const int at = len.ctx + k, tile = at / kKeys;
            if (!((mask >> k) & 1ull) || tile < cur.first || tile >= cur.first + tiles) continue;
            if (!DSPARK_CHECK(at / p.page < p.max_blocks && cur.b < p.B)) continue;
            const int block = p.table[cur.b * p.table_ld + at / p.page];
            if (block < 0 || block >= p.n_blocks) continue;
            const T* from = static_cast<const T*>(p.v) + block * p.block_stride +
                            (int64_t)(at % p.page) * p.token_stride + cur.head * p.head_stride +
                            c * 32;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t bits = __ldg(reinterpret_cast<const unsigned short*>(from) + j);
              if (any_special<T>(bits)) v[j] += H::widen(bits);
            }
          }
        }
        if (mine && full && DSPARK_CHECK(row_held(p, to))) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to * D + c * 32);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            out[j] = make_uint4(H::pack(v[8 * j] * inv, v[8 * j + 1] * inv),
                                H::pack(v[8 * j + 2] * inv, v[8 * j + 3] * inv),
                                H::pack(v[8 * j + 4] * inv, v[8 * j + 5] * inv),
                                H::pack(v[8 * j + 6] * inv, v[8 * j + 7] * inv));
        } else if (mine && DSPARK_CHECK(!full && part_held(p, slot, part_row))) {
          constexpr int kWide = W::kPartWide;
          float* out = part_at(ws, slot, p.part_rows, kWide, part_row, D, c * 32);
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             out + j / kWide * (p.part_rows * kWide) + j % kWide),
                         "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3]), "f"(v[j + 4]),
                         "f"(v[j + 5]), "f"(v[j + 6]), "f"(v[j + 7])
                         : "memory");
        }
        __syncwarp();
      }
      if (mine && DSPARK_CHECK(full ? row_held(p, to) : part_held(p, slot, part_row))) {
        if (!full)
          ws.stats[slot + part_row] = make_float2(ref, sum);
        else if (p.lse)
          p.lse[to] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      }
      tc_before_sync();  // the accumulators are read: the next item may take them
      cur = ahead;
    }
  } else if (warp < 10) {
    // ------------------------------------------------------ keys and values
    // Lane i copies the tile's box i, a part of one block.  Under kPair a warp
    // copies the keys and the values of its stream, else warp 8 copies the
    // keys and warp 9 the values.
    const int x = kPaired ? warp - 8 : 0;
    const bool keys = kPaired || warp == 8, values = kPaired || warp == 9;
    WideStream& stream = sh.stream[x];
    const uint32_t k_at = ring + x * W::kRing, v_at = k_at + kStages * W::kTileBytes;
    const int k_rows = boxes.k_rows, v_rows = boxes.v_rows;  // powers of two, k_rows at most v_rows
    const int v_boxes = kKeys / v_rows;
    const int rows = keys ? k_rows : v_rows, n_boxes = kKeys / rows;  // at most 16
    const uint32_t all_boxes = (1u << n_boxes) - 1u;
    const int v_lane = lane * v_rows / rows & 31;  // the box where this lane's values begin
    const int k_shift = 31 - __clz(k_rows);
    const int next_row = kKeys % p.page, next_block = kKeys / p.page;  // from tile to tile
    uint32_t g = 0, k_tiles = 0, v_tiles = 0;  // k_tiles, v_tiles: the tiles copied
    bool ok = !DSPARK_STALLED(blockIdx.x);
    Walk cur = walk_from(p, sh.start[x], ranges[x], p.item_cost);
    while (ok && cur.advance(p, kKeys)) {
      const int tiles = cur.count;
      const Lengths len = cur.len;
      const int first = cur.first * kKeys;
      // the place of this lane's box: position, entry of the table, row of the block
      int pos = first + lane * rows, at = pos / p.page, row_ahead = pos - at * p.page;
      const int32_t* table = p.table + cur.b * p.table_ld;
      auto entry = [&]() -> int {
        return lane < n_boxes && pos < len.len &&
                       DSPARK_CHECK(at == pos / p.page && at < p.max_blocks && cur.b < p.B)
                   ? __ldg(table + at)
                   : -1;
      };
      int ahead = entry();
      for (int i = 0; i < tiles; ++i, ++g) {
        const int block = ahead, row_here = row_ahead;
        pos += kKeys;
        at += next_block;
        row_ahead += next_row;
        if (row_ahead >= p.page) {
          row_ahead -= p.page;
          ++at;
        }
        ahead = entry();
        const bool held = block >= 0 && block < p.n_blocks;
        const int from = held ? block : p.n_blocks, row = held ? row_here : 0;
        const uint32_t stage = g % kStages;
        if (keys) {
          const uint32_t held_boxes = __ballot_sync(0xffffffffu, held);
          ok = wait_all(&stream.k_empty[stage], phase_of(g) ^ 1u);
          if (!ok) break;
          if (lane < kKeys / 32) {
            uint32_t word = ~0u;  // positions 32 lane .. of the tile
            if (held_boxes != all_boxes) {
              const uint32_t mine = held_boxes >> (lane << 5 >> k_shift);
              word = 0u;
              if (k_rows >= 32) {
                word = mine & 1u ? ~0u : 0u;
              } else {
                for (int j = 0; j << k_shift < 32; ++j)
                  if ((mine >> j) & 1u) word |= ((1u << k_rows) - 1u) << (j << k_shift);
              }
            }
            const int past = len.len - (first + i * kKeys + lane * 32);  // positions before the end
            stream.valid[g & 7u][lane] =
                past >= 32 ? word : past > 0 ? word & ((1u << past) - 1u) : 0u;
          }
          __syncwarp();  // lane 0's arrival stands for both lanes' words
          if (lane == 0) {
            stream.special[g & 7u] = 0u;
            mbar_arrive_expect_tx(&stream.k_full[stage], W::kTileBytes);
          }
          __syncwarp();
          // rows of one block, and a place inside the stage
          if (lane < n_boxes && DSPARK_CHECK(row + k_rows <= p.page && cur.head < p.kv_heads &&
                                             lane * (boxes.k_whole ? k_group : k_rows * 128u) +
                                                     (boxes.k_whole ? k_group : k_rows * 128u) <=
                                                 (boxes.k_whole ? W::kTileBytes : k_half) &&
                                             stage < kStages)) {
            const uint32_t to = k_at + stage * W::kTileBytes;
            if (boxes.k_whole) {
              tma_load_box(to + lane * k_group, &k_map, row, 0, cur.head, from,
                           &stream.k_full[stage]);
            } else {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_box(to + h * k_half + lane * k_rows * 128, &k_map, row, h, cur.head, from,
                             &stream.k_full[stage]);
            }
          }
          k_tiles = g + 1u;
          __syncwarp();
        }
        if (values) {
          const int v_from = kPaired ? __shfl_sync(0xffffffffu, from, v_lane) : from;
          const int v_row = kPaired ? __shfl_sync(0xffffffffu, row, v_lane) : row;
          ok = wait_all(&stream.v_empty[stage], phase_of(g) ^ 1u);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&stream.v_full[stage], W::kTileBytes);
          __syncwarp();
          if (lane < v_boxes && DSPARK_CHECK(v_row + v_rows <= p.page && cur.head < p.kv_heads &&
                                             (lane + 1) * v_box <= W::kTileBytes))
            tma_load_box(v_at + stage * W::kTileBytes + lane * v_box, &v_map, v_row, 0, cur.head,
                         v_from, &stream.v_full[stage]);
          v_tiles = g + 1u;
          __syncwarp();
        }
      }
    }
    // no copy is in flight when the CTA ends, which only a wait that expired can leave
    for (uint32_t i = 0; i < kStages; ++i) {
      if (i < k_tiles)
        mbar_wait_bounded(&stream.k_full[(k_tiles - 1u - i) % kStages], phase_of(k_tiles - 1u - i));
      if (i < v_tiles)
        mbar_wait_bounded(&stream.v_full[(v_tiles - 1u - i) % kStages], phase_of(v_tiles - 1u - i));
    }
  } else if (warp >= 10 && warp < 10 + (kPaired ? 2 : n_tiles)) {
    // ------------------------------------------------------------- products
    // A warp for each row tile, so that one's waits pass during the other's
    // products.  Under kBoth the two take turns, tile by tile: products of both
    // issued side by side would end together, and both warps would wait then.
    // The warp goes through the loop together; one lane issues.
    const int m = warp - 10;
    const int x = kPaired ? m : 0;
    WideStream& stream = sh.stream[x];
    constexpr uint32_t kFormat = H::kExponent == 0x7F80u ? 1u : 0u;  // bf16 or f16
    // fp32 accumulators, both operands of T, 128 rows; for P V the second has its dims outermost
    constexpr uint32_t kCommon = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (8u << 24);
    constexpr uint32_t kScores = kCommon | ((uint32_t)(kKeys / 8) << 17);
    constexpr uint32_t kValues = kCommon | (1u << 16) | ((uint32_t)(D / 8) << 17);
    const bool on = elect_one();
    // descriptors of this row tile of Q, and of the stages of keys and values; an operand further
    // on adds its distance / 16
    const uint64_t q_desc = operand_desc(base + m * W::kQBytes, 16, 1024);
    const uint64_t k_desc = operand_desc(ring + x * W::kRing, 16, k_group);
    const uint64_t v_desc = operand_desc(ring + x * W::kRing + kStages * W::kTileBytes, v_half,
                                         boxes.v_rows == 8 ? v_box : 1024u);
    // a tile's values, 16 positions after 16: within a box, or in the next ones
    uint64_t v_at[kKeys / 16];
#pragma unroll
    for (int kt = 0; kt < kKeys / 16; ++kt) {
      const int r = kt * 16;
      v_at[kt] = v_desc + (r / boxes.v_rows * v_box + r % boxes.v_rows * 128) / 16;
    }
    const uint32_t k_half16 = k_half / 16;
    const bool turns = kMode == kBoth && n_tiles == 2;
    auto scores = [&](uint32_t g, bool pass) {  // pass: gives the turn away
      const uint64_t b = k_desc + (g % kStages) * (W::kTileBytes / 16);
#pragma unroll
      for (int kt = 0; kt < D / 16; ++kt) {
        mma_ss(on, s_col(m, g), q_desc + (kt >> 2) * (16384 / 16) + (kt & 3) * 2,
               b + (kt >> 2) * k_half16 + (kt & 3) * 2, kScores, kt > 0);
        // half the products take as long as the other warp needs to see it
        if (kt == D / 32 - 1 && pass) mbar_arrive(&sh.turn[m ^ 1]);
      }
      mma_commit(on, &sh.s_full[m][g % W::kScores]);
      mma_commit(on, &stream.k_empty[g % kStages]);
    };
    auto values = [&](uint32_t g, bool add) {
      const uint64_t stage = (g % kStages) * (W::kTileBytes / 16);
#pragma unroll
      for (int kt = 0; kt < kKeys / 16; ++kt)
        mma_ts(on, o_col(m), s_col(m, g) + kt * 8, v_at[kt] + stage, kValues, add || kt > 0);
      mma_commit(on, &sh.o_full[m][g & 1u]);
      mma_commit(on, &stream.v_empty[g % kStages]);
    };
    uint32_t g = 0, segments = 0;
    bool ok = true;
    Walk cur = walk_from(p, sh.start[x], ranges[x], p.item_cost);
    while (ok && cur.advance(p, kKeys)) {
      const int tiles = cur.count;
      ok = wait_all(&sh.q_full[m], segments & 1u);
      for (int i = 0; i < min(W::kScores, tiles) && ok; ++i) {
        ok = wait_all(&stream.k_full[(g + i) % kStages], phase_of(g + i));
        if (!ok) break;
        tc_after_sync();
        scores(g + i, false);
      }
      for (int i = 0; i < tiles && ok; ++i, ++g) {
        const uint32_t ahead = g + W::kScores;  // takes the place of tile g's scores
        const bool more = i + W::kScores < tiles;
        // The weights, the values, where their copies run ahead of the scores the next keys, and
        // the turn (the values again where there is none: the barrier of keys read before may have
        // gone on).  The second row tile's turn also says that the first has cleared the values.
        constexpr bool kEarly = kStages > W::kScores;
        uint64_t* v_full = &stream.v_full[g % kStages];
        const uint32_t v_phase = phase_of(g);
        ok = wait_each({&sh.p_full[m][g % W::kScores], v_full,
                        kEarly && more ? &stream.k_full[ahead % kStages] : v_full,
                        turns ? &sh.turn[m] : v_full},
                       {score_phase(g), v_phase, kEarly && more ? phase_of(ahead) : v_phase,
                        turns ? (g + 1u + m) & 1u : v_phase});
        if (!ok) break;
        tc_after_sync();
        values(g, i > 0);
        if (more) {
          if constexpr (!kEarly) {
            ok = wait_all(&stream.k_full[ahead % kStages], phase_of(ahead));
            if (!ok) break;
          }
          scores(ahead, turns);
        } else if (turns) {
          mbar_arrive(&sh.turn[m ^ 1]);
        }
      }
      ++segments;
    }
    // nothing of this row tile's is in flight when its memory is given back
    mma_commit(on, &sh.drained[m]);
    mbar_wait_bounded(&sh.drained[m], 0);
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  if (warp == 10) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  // After a wait that expired the requests of the range are refused.  What the CTA has written of
  // them may be unfinished: NaN takes its place, and in the parts the joining kernel's sums.
  if (!sh.failed) return;
  for (int x = 0; x < W::kStreams; ++x) {
    if (ranges[x] <= 0) continue;
    Walk cur = walk_from(p, sh.start[x], ranges[x], p.item_cost);
    Lost lost = {cur.b, -1};
    while (cur.advance(p, kKeys)) {
      lost.last = cur.b;
      const int64_t slot = cur.slot(blockIdx.x * W::kStreams + x) * p.part_rows;
      for (int r = tid; r < min(W::kRows, p.nodes * p.group - r0); r += kWideThreads) {
        const int node = (r0 + r) / p.group;
        const int64_t to = ((int64_t)cur.b * p.nodes + node) * p.heads + cur.head * p.group + r0 +
                           r - node * p.group;
        if (!DSPARK_CHECK(cur.whole() ? row_held(p, to) : part_held(p, slot, r))) continue;
        if (!cur.whole()) {
          ws.stats[slot + r] = make_float2(NAN, NAN);
          continue;
        }
        for (int d = 0; d < D; d += 2)
          *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + to * D + d) = H::pack(NAN, NAN);
        if (p.lse) p.lse[to] = NAN;
      }
    }
    if (tid == 0 && DSPARK_CHECK(blockIdx.x * W::kStreams + x < p.max_ctas))
      ws.lost[blockIdx.x * W::kStreams + x] = lost;
  }
}

// rows of a tensor copy: the most that divide a block and a tile; the swizzle
// wants whole groups of eight
inline int wide_box_rows(int page, int keys) {
  int rows = keys;
  while (page % rows) rows /= 2;
  return rows;
}

// the map of one cache: 64 dims, rows of a block, blocks of 64 dims, heads, blocks
template <typename T>
bool map_cache(CUtensorMap* map, const Params& p, const void* cache, int dim, int box_rows,
               bool whole) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t sizes[5] = {64, (cuuint64_t)p.page, (cuuint64_t)dim / 64,
                               (cuuint64_t)p.kv_heads, (cuuint64_t)p.n_blocks};
  const cuuint64_t strides[4] = {(cuuint64_t)p.token_stride * 2, 128,
                                 (cuuint64_t)p.head_stride * 2, (cuuint64_t)p.block_stride * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, whole ? (cuuint32_t)dim / 64 : 1u, 1, 1};
  const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
  return encode(map,
                Half<T>::kExponent == 0x7F80u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                5, const_cast<void*>(cache), sizes, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// false: the cache's shape has no map, or blocks not made of groups of eight
template <typename T, int D, WideMode kMode>
bool launch_wide(Params p, int sms, cudaStream_t stream, cudaError_t* error) {
  using W = Wide<D, kMode>;
  const int rows = wide_box_rows(p.page, W::kKeys);
  if (rows < 8) return false;
  Boxes boxes;
  boxes.k_whole = W::kKeys / rows * W::kHalves > W::kKeys / 8;
  boxes.k_rows = boxes.k_whole ? 8 : rows;
  boxes.v_rows = rows;
  CUtensorMap k_map, v_map;
  if (!map_cache<T>(&k_map, p, p.k, D, boxes.k_rows, boxes.k_whole) ||
      !map_cache<T>(&v_map, p, p.v, D, boxes.v_rows, true))
    return false;
  p.row_tiles = (p.nodes * p.group + W::kRows - 1) / W::kRows;
  p.part_rows = part_rows(p.nodes * p.group, W::kRows);
  p.part_wide = W::kPartWide;
  p.max_ctas = wide_ctas(kMode == kPair);
  p.tile = W::kKeys;
  p.waits = true;
  p.item_cost = kMode == kPair ? kPairCost : kMode == kBoth ? kBothCost : kOneCost;
  auto* kernel = tree_attention_wide_kernel<T, D, kMode>;
  *error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
  if (*error != cudaSuccess) return true;
  const int grid = min(p.max_ctas / W::kStreams, max(sms, p.row_tiles));
  kernel<<<grid, kWideThreads, W::kSmem, stream>>>(p, k_map, v_map, boxes);
  *error = cudaGetLastError();
  if (*error == cudaSuccess)
    *error = launch_join<T, D>(p, W::kRows, grid * W::kStreams, stream);
  return true;
}

// The streaming kernel for few rows, whose products need no tensor memory and
// whose two to four CTAs per SM hide one another's starts, and for blocks that have no
// tensor copies; else the tensor kernel.
template <typename T, int D>
cudaError_t launch_dim(const Params& p, int sms, cudaStream_t stream) {
  const int rows = p.nodes * p.group, shape = stream_rows(rows, D);
  cudaError_t e;
  if constexpr (D == 256) {
    if (launch_wide<T, D, kOne>(p, sms, stream, &e)) return e;
    if (shape == 8) return launch_shape<T, D, 1, 1>(p, sms, stream);
    if (shape == 16) return launch_shape<T, D, 2, 1>(p, sms, stream);
    return launch_shape<T, D, 2, 4>(p, sms, stream);
  } else {
    if (rows > 128) {
      if (launch_wide<T, D, kBoth>(p, sms, stream, &e)) return e;
    } else if (rows > few_rows(D)) {
      if (launch_wide<T, D, kPair>(p, sms, stream, &e)) return e;
    }
    if (shape == 8) return launch_shape<T, D, 1, 1>(p, sms, stream);
    if (shape == 16) return launch_shape<T, D, 2, 1>(p, sms, stream);
    if (shape == 24) return launch_shape<T, D, 3, 1>(p, sms, stream);
    if (shape == 32) return launch_shape<T, D, 4, 1>(p, sms, stream);
    return launch_shape<T, D, 4, 2>(p, sms, stream);
  }
}

}  // namespace attn
}  // namespace dspark
