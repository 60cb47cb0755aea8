// latent_attention.cuh -- the kernels of dspark_latent_attention.  Division of
// work, walk along it and workspace are those of tree_attention.cuh, with an
// item for each (request, tile of 128 rows).
#pragma once

#include "tree_attention_wide.cuh"

namespace dspark {
namespace attn {

struct LatentParams : Params {
  int latent, width;  // of a row of the cache: its values, all of it
};

// ------------------------------------------- a pair of CTAs and its barriers
// The address of this CTA's shared address `addr` in CTA `rank` of the pair.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void cluster_fence() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void pair_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Tensor copies into this CTA that complete on a barrier of either; what lies beyond the map is 0.
// From element x of row r of block b (or of request b of Q):
__device__ __forceinline__ void pair_load_box(uint32_t dst, const CUtensorMap* map, int x, int r,
                                              int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(r), "r"(b), "r"(bar)
      : "memory");
}
// several chunks of 64 elements, from chunk c on
__device__ __forceinline__ void pair_load_chunks(uint32_t dst, const CUtensorMap* map, int r, int c,
                                                 int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(r), "r"(c), "r"(b), "r"(bar)
      : "memory");
}
// d (+)= a b over the pair, a's rows and b's columns from both CTAs' shared memory
__device__ __forceinline__ void pair_mma(bool on, uint32_t d, uint64_t a, uint64_t b,
                                         uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"((uint32_t)on)
      : "memory");
}
// arrives on `bar` in both CTAs once every product issued before it is done
__device__ __forceinline__ void pair_commit(bool on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %2;\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)on), "h"((uint16_t)3)
      : "memory");
}
// whether any of the 256 softmax threads says so; all of them call
__device__ __forceinline__ bool any_of_256(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred.aligned q, 1, 256, "
      "p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0u;
}

// The rest of a bounded wait of a whole warp, out of its callers' loops.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t phase, uint32_t* failed) {
  const uint64_t t0 = global_ns();
  uint32_t nap = 32;
  while (!__any_sync(0xffffffffu, *(volatile uint32_t*)failed)) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
    if (__any_sync(0xffffffffu, global_ns() - t0 >= kWaitLimitNs)) {
      *(volatile uint32_t*)failed = 1u;
      break;
    }
    if (nap > 32u) __nanosleep(nap);
    nap = nap < 1024u ? 2u * nap : 1024u;
  }
  return false;
}

// ------------------------------------------------------------ the kernel
// A pair of CTAs takes 128 rows of an item, 64 a CTA, and goes over the keys
// in tiles of 128 positions.  512 dims of fp32 accumulators for 128 rows
// would fill the tensor memory of one SM; with products of the pair
// (cta_group::2, 128 rows) a CTA's 64 rows take its 128 lanes twice: half of
// a product's columns in lanes 0-63, the other half in lanes 64-127, so that
// 64 columns hold the scores of 128 positions and 256 the accumulators, at
// the full rate (32 cycles a product of 128 columns, 64 of 256).
//
// S = Q K^T: each CTA brings its 64 rows of Q and 64 of the tile's rows of
// the cache, in groups of three chunks of 64 elements (24 KB) that are freed
// one by one.  O += P V: each CTA brings its rows' weights (through shared
// memory) and its half of the values' dims for all 128 positions, in pieces
// of 64 positions; a row's values are its keys' first elements, but half of
// them belong to the other CTA, so they are copied again (from L2).  The
// scores of the next tile are computed before the values of this one, while
// the softmax of this one runs; its weights are handed over by halves of the
// positions, as the products free their place by halves.
//
// Warps 0-7: softmax; a thread has a row's scores of 32 positions, so four
// threads share a row: the threads vote whether any score passes its row's
// reference by more than 8, and only then exchange maxima and rescale.  Also
// results.  Warp 8: tensor copies of keys; warp 9: of queries and values.  Warps
// 10 and 11 of CTA 0 issue the pair's products.
//
// A tile's 52 products take 2,192 cycles, its softmax 1,600; it takes about
// 3,000 in the loop: the issuing warps' waits (200 cycles each), the softmax
// between a tile's scores and its values, and the copies' latency behind a
// ring of one tile.  Two requests of 120,000 tokens and 192 rows 104 us (256
// rows' products, 1.3 PFLOP/s), 64 of 4,000 and 96 rows 74 us (4.2 TB/s), of
// which 7 us pass before the first keys, 5 behind the last product and 5 to 10
// in the join.  A request's tiles of rows are counted from the batch's nodes:
// those without a node of the request's cost as much as full ones (16 requests
// of 2,500 to 8,100 tokens, 32 heads, 24 nodes 109 us; with one node each 105,
// and 29 where the batch has one).  Slower or the same: cluster-scoped barrier operations (524 us
// where 217 were left), half the values through the load path by four more
// warps (112 -> 122 us), four chunks of Q in tensor memory and a longer ring
// instead (112 -> 113), unrolled product loops (107 -> 112: they fall out of the
// scheduler's instruction cache), the prefetch two tiles ahead (106 -> 112).
constexpr int kLatentKeys = 128;  // positions of a tile
// 168 registers a thread, 16 to 24 bytes of it spilled; from 416 threads on 128 and 146 to 314.
constexpr int kLatentThreads = 384;
// An item's cost in tiles, at 3, 4, 5, 6: 256 requests of mixed lengths and 128 rows 157, 157, 156,
// 158 us, 64 of 96 rows 57, 55, 55, 55, two long ones 107, 110, 114, 114 (at 2 all are 1 to 3 %
// slower than at 3).  The least of a range: one request of 717 tokens at 1, 2, 3, 4 takes 16.2,
// 16.3, 17.9, 18.6 us.
constexpr int kLatentCost = 3, kLatentMinRange = 2;

template <int DV>
struct Latent {
  static constexpr int kHalf = DV / 2;            // values' dims of a CTA
  static constexpr int kChunks = DV / 64 + 1;     // of 64 elements, of a row of the cache
  static constexpr int kGroup = 3;                // chunks that come together
  static constexpr int kKSlots = DV == 512 ? 3 : 4;
  static constexpr int kVSlots = DV == 512 ? 2 : 4;  // pieces of 64 positions
  static constexpr int kVParts = kHalf / 64;      // chunks of a piece
  static constexpr int kChunkBytes = 64 * 128;
  static constexpr int kKBytes = kGroup * kChunkBytes, kVBytes = kVParts * kChunkBytes;
  static constexpr int kQBytes = kChunks * kChunkBytes;
  static constexpr int kPBytes = 64 * kLatentKeys * 2;
  static constexpr int kSmem = kQBytes + kKSlots * kKBytes + kVSlots * kVBytes + kPBytes + 1024;
};

struct LatentShared {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full, q_empty, drained;
  // by tile number modulo 2: the scores are there; the first products of scores, of values are issued
  uint64_t s_full[2], s_turn[2], v_turn[2];
  // by half of a tile's positions: the weights are there (and by tile number modulo 2), have been
  // multiplied; the values are there for CTA 1 to look at
  uint64_t p_full[2][2], o_full[2], v_go[2];
  uint64_t scan[32];
  // by tile number modulo 16: a narrow row's keys are copied up to 7 tiles ahead of the results
  uint32_t valid[16][4];  // a tile's positions that hold a key
  uint32_t special[16];   // a value of a tile's nodes is an infinity or a NaN
  Start start;
  uint32_t tmem;
  uint32_t failed;  // a wait expired
  uint32_t peer_failed, issued[3], peer_issued[3];  // copies of keys, values, queries
};

// The maps of the tensor copies, and the shapes of their boxes.
struct LatentMaps {
  CUtensorMap tail;    // {elements, rows of a block, blocks}, a chunk of `rows` rows
  CUtensorMap keys;    // {64, rows of a block, whole chunks, blocks}, kGroup chunks of k_rows rows
  CUtensorMap values;  // the same, a CTA's values of `rows` rows
  CUtensorMap q;       // {elements, rows of a request, requests}, a chunk of 64 rows
  int rows;            // of a block that are copied together: 8, 16, 32 or 64
  // 64 or 8; 0: keys are copied chunk by chunk.  64 requests of 4,000 tokens, 96 rows, in blocks of
  // 8, 16, 32, 64 tokens: by chunks 114, 82, 75, 75 us, by eight rows 78, 77, 77, 77, by 64 rows 74.
  int k_rows;
  // Q has a map (else the softmax warps copy it, 74 -> 81 us)
  int q_copies;
};

template <typename T, int DV>
__global__ void __launch_bounds__(kLatentThreads, 1) __cluster_dims__(2, 1, 1)
    latent_attention_kernel(const __grid_constant__ LatentParams p,
                            const __grid_constant__ LatentMaps maps) {
  using H = Half<T>;
  using L = Latent<DV>;
  constexpr int kKeys = kLatentKeys;
  extern __shared__ unsigned char smem_raw[];
  __shared__ LatentShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const uint32_t q_at = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_at = q_at + L::kQBytes, v_at = k_at + L::kKSlots * L::kKBytes;
  const uint32_t p_at = v_at + L::kVSlots * L::kVBytes;
  const int chunks = (p.width + 63) / 64, groups = (chunks + L::kGroup - 1) / L::kGroup;
  const int all_rows = p.nodes * p.heads, rows = maps.rows;
  // Where a copied group of keys lies: runs of k_rows rows, each with its chunks one after the
  // other; chunk after chunk where it is copied so.  Values: runs of `rows` rows, each with its
  // chunks one after the other.
  const int whole_groups = maps.k_rows ? p.width / 64 / L::kGroup : 0;
  const uint32_t k_chunk = maps.k_rows == 8 ? 1024u : L::kChunkBytes;
  const uint32_t k_eight = maps.k_rows == 8 ? L::kGroup * 1024u : 1024u;  // rows
  const uint32_t v_chunk = rows * 128u, v_run = L::kVParts * v_chunk;
  const int shift = 31 - __clz(rows);  // a power of two

  if (tid < 4)
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<const CUtensorMap*>(&maps) + tid)
                 : "memory");
  if (tid == 0) {
    for (int i = 0; i < L::kKSlots; ++i) {
      mbar_init(&sh.k_full[i], 2);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < L::kVSlots; ++i) {
      mbar_init(&sh.v_full[i], 2);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.q_full, maps.q_copies ? 2 : 16);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_turn[i], 32);
      mbar_init(&sh.v_turn[i], 32);
      mbar_init(&sh.p_full[i][0], 8);
      mbar_init(&sh.p_full[i][1], 8);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.v_go[i], 1);
    }
    mbar_init(&sh.drained, 2);
    sh.failed = sh.peer_failed = 0u;
    for (int i = 0; i < 3; ++i) sh.issued[i] = sh.peer_issued[i] = 0u;
    mbar_init_fence();
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const Workspace ws = carve(p.workspace, p.part_rows, p.max_ctas);
  int64_t range;
  find_range<kLatentThreads, 1>(p, ws, sh.scan, &sh.start, &range, pair, pairs, rank == 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && rank == 0 && DSPARK_CHECK(pair < p.max_ctas)) ws.lost[pair] = {0, -1};
  tc_before_sync();
  __syncthreads();
  cluster_sync();
  tc_after_sync();
  const uint32_t tmem = sh.tmem;
  if (range <= 0) {  // both CTAs
    if (warp == 10)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    return;
  }
  auto s_col = [&](uint32_t g) -> uint32_t { return tmem + (g & 1u) * 64u; };
  const uint32_t o_col = tmem + 128u;

  // bounded waits of a whole warp, as in tree_attention_wide_kernel
  auto wait_all = [&](uint64_t* bar, uint32_t phase) -> bool {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, phase)) || wait_long(bar, phase, &sh.failed);
  };

  if (warp < 8) {
    // -------------------------------------------------- softmax and results
    const int t = tid & 127, wg = tid >> 7;   // lane of tensor memory; which columns
    const int row = t & 63, half = t >> 6;    // of this CTA's rows; positions and dims from 64, DV/2
    const int word = half * 2 + wg;           // this thread's 32 positions of a tile
    const uint32_t lanes = (uint32_t)(t & ~31) << 16;
    const uint32_t oc = o_col + wg * (DV / 4) + lanes;
    // as in tree_attention_wide_kernel: a negative scale goes into Q's sign
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;
    const float scale = fmaxf(fabsf(p.scale2), 1.17549435e-38f);
    const uint32_t q_full = in_cta(smem_u32(&sh.q_full), 0);
    const uint32_t p_full = in_cta(smem_u32(&sh.p_full[half][0]), 0);
    const uint32_t v_go = in_cta(smem_u32(&sh.v_go[half]), 1);
    const uint32_t special_there = in_cta(smem_u32(sh.special), rank ^ 1u);
    // four floats a row, in the place of the weights between two products
    const uint32_t exchange = p_at + row * 16;
    uint32_t tile_no = 0, goes = 0;
    bool bad = false;                            // a wait of this warp expired

    auto fill_q = [&](const Walk& w) {
      constexpr int kPieces = L::kChunks * 8, kEach = 64 * kPieces / 256, kBatch = kEach / 2;
      const int first = w.head * 128 + (int)rank * 64, live = w.len.nodes * p.heads;
      const T* from = static_cast<const T*>(p.q) + w.b * p.q_req;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint4 q[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = tid + (part * kBatch + i) * 256, r = at / kPieces, c = at % kPieces;
          q[i] = make_uint4(0u, 0u, 0u, 0u);
          if (first + r < live && c * 8 < p.width &&
              DSPARK_CHECK(w.b < p.B && first + r < all_rows)) {
            const int node = (first + r) / p.heads;
            q[i] = __ldg(reinterpret_cast<const uint4*>(
                from + node * p.q_node + (int64_t)(first + r - node * p.heads) * p.q_head + c * 8));
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = tid + (part * kBatch + i) * 256, r = at / kPieces, c = at % kPieces;
          const uint32_t to = q_at + (c >> 3) * L::kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          if (!DSPARK_CHECK(to + 16 <= k_at)) continue;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(q[i].x ^ flip),
                       "r"(q[i].y ^ flip), "r"(q[i].z ^ flip), "r"(q[i].w ^ flip)
                       : "memory");
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) pair_arrive(q_full);
    };
    // For the products with half h of tile g's weights, or with both.  The phase before has been
    // seen by this warp, or by one that has voted with it since: no phase is taken for another.
    auto wait_half = [&](int h, uint32_t g) {
      bad = bad || !wait_all(&sh.o_full[h], g & 1u);
      tc_after_sync();
    };
    auto wait_values = [&](uint32_t g) {
      wait_half(0, g);
      wait_half(1, g);
    };
    auto put = [&](float v) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(exchange + word * 4), "f"(v) : "memory");
    };
    auto get = [&]() -> float4 {
      float4 v;
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(exchange)
                   : "memory");
      return v;
    };
    // Whether one of the eight warps is lost: what each of them asks at the same barrier, so that
    // they leave together.
    auto lost = [&]() -> bool { return any_of_256(bad); };

    Walk cur = walk_from(p, sh.start, range, p.item_cost);
    bool more = cur.advance(p, kKeys), ok = true;
    if (more && !maps.q_copies) fill_q(cur);
    while (ok && more) {
      const int tiles = cur.count;
      const Lengths len = cur.len;
      const int live = len.nodes * p.heads;
      const int item_row = cur.head * 128 + (int)rank * 64 + row;
      if (tid == 0 && rank == 0 && cur.head == 0 && cur.first == 0)
        p.status[cur.b] = len.bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;
      Walk ahead = cur;
      more = ahead.advance(p, kKeys);
      const bool idle = item_row - (t & 31) >= live;  // no row of this warp has a node
      const int node = item_row / p.heads;
      uint64_t mask = 0;
      if (item_row < live && DSPARK_CHECK(node < p.nodes && cur.b < p.B))
        mask = p.mask ? p.mask[(int64_t)cur.b * p.nodes + node] : ~0ull >> (63 - node);
      float ref = -INFINITY;
      float2 sum2 = make_float2(0.0f, 0.0f);
      for (int i = 0; i < tiles; ++i, ++tile_no) {
        bad = bad || !wait_all(&sh.s_full[tile_no & 1u], (tile_no >> 1) & 1u);
        tc_after_sync();
        const int pos = (cur.first + i) * kKeys;
        const bool nodes_here = pos + kKeys > len.ctx;
        float v[32];
        float top = -INFINITY;
        if (!idle) {
          tmem_load32(v, s_col(tile_no) + wg * 32 + lanes);
          uint32_t w = sh.valid[tile_no & 15u][word];
          tmem_wait_load();
          tc_before_sync();
          if (nodes_here) {
            const int node0 = pos + word * 32 - len.ctx;  // the node of the first position
            if (node0 >= 0)
              w &= node0 < 64 ? (uint32_t)(mask >> node0) : 0u;
            else if (node0 > -32)
              w &= (uint32_t)(mask << -node0) | ((1u << -node0) - 1u);
          }
          if (__builtin_expect(!__all_sync(0xffffffffu, w == ~0u), 0)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((w >> j) & 1u)) v[j] = -INFINITY;
          }
          float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int j = 4; j < 28; j += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(fmaxf(m4[k], v[j + k]), v[j + 4 + k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], v[28 + k]);
          if (item_row < live) top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
        }
        bool waited = i == 0;  // for the products before, of which the weights' place is free
        if (__builtin_expect(any_of_256(bad || top > ref + kSlack), 0)) {
          if (!waited) wait_values(tile_no - 1u);
          waited = true;
          put(top);
          if (lost()) {
            ok = false;
            break;
          }
          const float4 tops = get();
          top = fmaxf(fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w)), ref);
          const float f = top == -INFINITY ? 1.0f : exp2_approx(ref - top);
          ref = top;
          sum2.x *= f;
          sum2.y *= f;
          if (i > 0 && !idle) {
#pragma unroll 1
            for (int c = 0; c < DV / 64; ++c) {
              uint32_t a[16];
              tmem_load16(a, oc + c * 16);
              tmem_wait_load();
#pragma unroll
              for (int j = 0; j < 16; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
              tmem_store16(oc + c * 16, a);
            }
            tmem_wait_store();
          }
          // The next product takes all lanes, and its first half waits for half of these warps only:
          // it is ordered behind the others' stores by this barrier.
          tc_before_sync();
          any_of_256(false);  // all have read before the weights take the place
          tc_after_sync();
        }
        uint32_t w16[16];
        if (!idle) {
          const float2 off = f2(ref == -INFINITY ? 0.0f : -ref), by = f2(scale);
          float2 part2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = fma2_rn(make_float2(v[2 * j], v[2 * j + 1]), by, off);
            e.x = exp2_approx(e.x);
            e.y = exp2_approx(e.y);
            if (j & 1)
              part2 = add2_rn(part2, e);
            else
              sum2 = add2_rn(sum2, e);
            w16[j] = H::pack(e.x, e.y);
          }
          sum2 = add2_rn(sum2, part2);
        }
        if (!waited) wait_half(half, tile_no - 1u);
        if (!idle) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             p_at + half * 8192 + row * 128 + (((wg * 4 + j) ^ (row & 7)) << 4)),
                         "r"(w16[4 * j]), "r"(w16[4 * j + 1]), "r"(w16[4 * j + 2]),
                         "r"(w16[4 * j + 3])
                         : "memory");
        }
        if (__builtin_expect(nodes_here, 0)) {
          // Rows from the first node on, which some rows see and others do not, and what lies
          // behind the end: infinities and NaN are cleared, as 0 times them would reach rows that
          // do not see them.  CTA 1 learns from CTA 0 that its values are there.
          // Each half's threads clear the positions that their weights belong to.
          const uint32_t piece = tile_no * 2u + half, slot = piece % L::kVSlots;
          if (rank == 0) {
            bad = bad || !wait_all(&sh.v_full[slot], (piece / L::kVSlots) & 1u);
            if (t == half * 64 && wg == 0) {
              cluster_fence();
              pair_arrive(v_go);
            }
          } else {
            bad = bad || !wait_all(&sh.v_go[half], goes & 1u);
            cluster_fence();
          }
          ++goes;
          const int from = max(0, len.ctx - pos - half * 64);
          // blocks' rows that the last copy brought; zeros behind them
          const int end = min(64, (len.len - pos - half * 64 + rows - 1) & -rows);
          constexpr int kPer = L::kHalf / 8;  // 16-byte pieces of a position
          for (int j = wg * 64 + row; j < (end - from) * kPer && !bad; j += 128) {
            const int r = from + j / kPer, c = j % kPer;
            const uint32_t addr = v_at + slot * L::kVBytes + (r >> shift) * v_run +
                                  (c >> 3) * v_chunk + (r & (rows - 1)) * 128 +
                                  (((c & 7) ^ (r & 7)) << 4);
            if (!DSPARK_CHECK(addr >= v_at && addr + 16 <= p_at)) continue;
            uint32_t x[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(addr)
                         : "memory");
            if (any_special<T>(x[0]) || any_special<T>(x[1]) || any_special<T>(x[2]) ||
                any_special<T>(x[3])) {
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                           "r"(without_special<T>(x[0])), "r"(without_special<T>(x[1])),
                           "r"(without_special<T>(x[2])), "r"(without_special<T>(x[3]))
                           : "memory");
              if (pos + half * 64 + r < len.len) {
                *(volatile uint32_t*)&sh.special[tile_no & 15u] = 1u;
                pair_store(special_there + (tile_no & 15u) * 4, 1u);
                cluster_fence();
              }
            }
          }
        }
        fence_async_shared();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive(p_full + (tile_no & 1u) * 8u);
      }
      if (!ok) break;
      // Q is free, as the last scores are done
      if (more && !maps.q_copies) fill_q(ahead);
      if (lost()) break;
      wait_values(tile_no - 1u);
      float sum = sum2.x + sum2.y;
      if (item_row >= live) {  // a row of no node: its zero query saw the text all the same
        ref = -INFINITY;
        sum = 0.0f;
      }
      put(sum);
      if (lost()) break;
      const float4 sums = get();
      sum = (sums.x + sums.y) + (sums.z + sums.w);
      bool special = false;
      for (uint32_t k = 1; k <= min(2, tiles); ++k)
        special |= *(volatile uint32_t*)&sh.special[(tile_no - k) & 15u] != 0u;

      const bool mine = item_row < all_rows, full = cur.whole();
      const int64_t to = (int64_t)cur.b * all_rows + item_row;
      const int64_t slot = cur.slot(pair) * p.part_rows;
      const int part_row = (int)rank * 64 + row;
      const float inv = sum == 0.0f ? 0.0f : full ? 1.0f / sum : 1.0f;
      const int d0 = half * L::kHalf + wg * (DV / 4);  // this thread's dims
      const int pieces = item_row - (t & 31) < all_rows ? DV / 128 : 0;
      const uint32_t staged = p_at + warp * 2048;  // 32 rows of 64 bytes, swizzled
      if (full) any_of_256(false);  // all have read the sums, in whose place results are staged
#pragma unroll 1
      for (int c = 0; c < pieces; ++c) {
        const int d = d0 + c * 32;
        if (d >= p.latent) break;  // of the whole warp
        float v[32];
        tmem_load32(v, oc + c * 32);
        tmem_wait_load();
        if (item_row >= live) {
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
            const T* from = static_cast<const T*>(p.k) + block * p.block_stride +
                            (int64_t)(at % p.page) * p.token_stride + d;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t bits = __ldg(reinterpret_cast<const unsigned short*>(from) + j);
              if (any_special<T>(bits)) v[j] += H::widen(bits);
            }
          }
        }
        if (full) {
          // turned in shared memory, so that four lanes write 64 bytes of a row
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             staged + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                         "r"(H::pack(v[8 * j] * inv, v[8 * j + 1] * inv)),
                         "r"(H::pack(v[8 * j + 2] * inv, v[8 * j + 3] * inv)),
                         "r"(H::pack(v[8 * j + 4] * inv, v[8 * j + 5] * inv)),
                         "r"(H::pack(v[8 * j + 6] * inv, v[8 * j + 7] * inv))
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = k * 8 + (lane >> 2), j = lane & 3, there = item_row - lane + r;
            uint4 x;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(staged + r * 64 + ((j ^ ((r >> 1) & 3)) << 4))
                         : "memory");
            if (there < all_rows && DSPARK_CHECK(row_held(p, to - lane + r) && d + 32 <= p.latent))
              *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (to - lane + r) * p.latent + d +
                                        j * 8) = x;
          }
        } else if (mine && DSPARK_CHECK(part_held(p, slot, part_row))) {
          float* out = ws.rows + (slot + part_row) * DV + d;
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + j),
                         "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3]), "f"(v[j + 4]),
                         "f"(v[j + 5]), "f"(v[j + 6]), "f"(v[j + 7])
                         : "memory");
        }
        __syncwarp();
      }
      if (mine && word == 0 && DSPARK_CHECK(full ? row_held(p, to) : part_held(p, slot, part_row))) {
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
    // Lane i holds the place of the tile's i-th run of `rows` rows of one block.  Of a copy chunk by
    // chunk, lane i takes run i % per_half of 64 positions and chunk i / per_half; of a copy of
    // whole groups or of values, the lanes before per_half or 64 / k_rows take a run each.
    const bool keys = warp == 8;
    const int runs = kKeys / rows, per_half = runs / 2;  // powers of two, at most 16 and 8
    const int half_shift = 31 - __clz(per_half);
    const int next_row = kKeys % p.page, next_block = kKeys / p.page;
    const uint32_t all_runs = (1u << runs) - 1u;
    const int run = lane & (per_half - 1), chunk = lane >> half_shift;
    // boxes of eight rows: this lane's run, and its first row there
    const int eight = lane & 7, eight_run = eight * 8 >> shift, eight_row = eight * 8 & (rows - 1);
    const uint32_t k_full = in_cta(smem_u32(sh.k_full), 0), v_full = in_cta(smem_u32(sh.v_full), 0);
    const bool dense = p.token_stride == p.width;  // runs lie in one piece
    uint32_t g = 0, issued = 0, slot = 0, phase = 0, segments = 0;
    bool ok = !DSPARK_STALLED(blockIdx.x);
    Walk cur = walk_from(p, sh.start, range, p.item_cost);
    while (ok && cur.advance(p, kKeys)) {
      if (!keys && maps.q_copies) {
        // the item's queries, once the scores of the item before are done, which is before any
        // place of values is free
        ok = wait_all(&sh.q_empty, (segments & 1u) ^ 1u);
        if (!ok) break;
        const uint32_t bar = in_cta(smem_u32(&sh.q_full), 0);
        if (lane == 0) pair_arrive_expect_tx(bar, chunks * L::kChunkBytes);
        __syncwarp();
        if (lane < chunks && DSPARK_CHECK(cur.b < p.B && cur.head < p.kv_heads && lane < L::kChunks))
          pair_load_box(q_at + lane * L::kChunkBytes, &maps.q, lane * 64,
                        cur.head * 128 + (int)rank * 64, cur.b, bar);
        ++segments;
        __syncwarp();
      }
      const int tiles = cur.count;
      const Lengths len = cur.len;
      int pos = cur.first * kKeys + lane * rows, at = pos / p.page, row_ahead = pos - at * p.page;
      const int32_t* table = p.table + cur.b * p.table_ld;
      auto entry = [&]() -> int {
        return lane < runs && pos < len.len &&
                       DSPARK_CHECK(at == pos / p.page && at < p.max_blocks && cur.b < p.B)
                   ? __ldg(table + at)
                   : -1;
      };
      int ahead = entry();
      for (int i = 0; i < tiles && ok; ++i, ++g) {
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
        if (keys) {
          const uint32_t held_runs = __ballot_sync(0xffffffffu, held);
          const int at_run = (int)rank * per_half;
          const int b = __shfl_sync(0xffffffffu, from, at_run + run);
          const int r = __shfl_sync(0xffffffffu, row, at_run + run);
          const int b8 = __shfl_sync(0xffffffffu, from, at_run + eight_run);
          const int r8 = __shfl_sync(0xffffffffu, row, at_run + eight_run) + eight_row;
          if (lane < 4) {
            uint32_t word = ~0u;  // positions 32 lane .. of the tile
            if (held_runs != all_runs) {
              const uint32_t mine = held_runs >> (lane << 5 >> shift);
              word = 0u;
              if (rows >= 32) {
                word = mine & 1u ? ~0u : 0u;
              } else {
                for (int j = 0; j << shift < 32; ++j)
                  if ((mine >> j) & 1u) word |= ((1u << rows) - 1u) << (j << shift);
              }
            }
            const int past = len.len - ((cur.first + i) * kKeys + lane * 32);
            sh.valid[g & 15u][lane] = past >= 32 ? word : past > 0 ? word & ((1u << past) - 1u) : 0u;
          }
          if (lane == 0) sh.special[g & 15u] = 0u;
          __syncwarp();  // lane 0's arrivals stand for all lanes' words
          for (int x = 0; x < groups; ++x) {
            const int c = x * L::kGroup, here = min(L::kGroup, chunks - c);
            const uint32_t bar = k_full + slot * 8u, to = k_at + slot * L::kKBytes;
            ok = wait_all(&sh.k_empty[slot], phase ^ 1u);
            if (!ok) break;
            if (lane == 0) pair_arrive_expect_tx(bar, here * L::kChunkBytes);
            if (!DSPARK_CHECK(r + rows <= p.page && slot < L::kKSlots && r8 + 8 <= p.page)) {
            } else if (x < whole_groups) {
              if (maps.k_rows == 8) {
                if (lane < 8) pair_load_chunks(to + lane * k_eight, &maps.keys, r8, c, b8, bar);
              } else if (lane == 0) {
                pair_load_chunks(to, &maps.keys, r, c, b, bar);
              }
            } else if (chunk < here) {
              pair_load_box(to + chunk * L::kChunkBytes + run * rows * 128, &maps.tail,
                            (c + chunk) * 64, r, b, bar);
            }
            ++issued;
            if (++slot == L::kKSlots) slot = 0, phase ^= 1u;
            __syncwarp();
          }
          // The next tile's rows on their way to L2: the ring holds one tile, and an HBM latency
          // more from a place's release to its next keys would show.
          if (dense && lane >= at_run && lane < at_run + per_half && ahead >= 0 &&
              ahead < p.n_blocks && DSPARK_CHECK(row_ahead + rows <= p.page))
            l2_prefetch_bulk(static_cast<const T*>(p.k) + ahead * p.block_stride +
                                 (int64_t)row_ahead * p.token_stride,
                             rows * p.width * 2);
          __syncwarp();
        } else {
          for (int s = 0; s < 2; ++s) {  // 64 positions
            const int b = __shfl_sync(0xffffffffu, from, s * per_half + run);
            const int r = __shfl_sync(0xffffffffu, row, s * per_half + run);
            const uint32_t bar = v_full + slot * 8u;
            ok = wait_all(&sh.v_empty[slot], phase ^ 1u);
            if (!ok) break;
            if (lane == 0) pair_arrive_expect_tx(bar, L::kVBytes);
            if (lane < per_half && DSPARK_CHECK(r + rows <= p.page && slot < L::kVSlots &&
                                                (run + 1) * v_run <= L::kVBytes))
              pair_load_chunks(v_at + slot * L::kVBytes + run * v_run, &maps.values, r,
                               (int)rank * L::kVParts, b, bar);
            ++issued;
            if (++slot == L::kVSlots) slot = 0, phase ^= 1u;
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) {
      sh.issued[warp - 8] = issued;
      if (!keys) sh.issued[2] = segments;
    }
  } else if (rank == 0) {
    // ------------------------------------------------------------- products
    // A warp for the scores and one for the values, so that one's waits, 200 cycles each where the
    // tensor cores hold some 100 cycles of products ahead, pass during the other's products.  They
    // take turns: tile g's scores behind the first half of tile g - 2's values, and tile g's values
    // behind tile g + 1's scores (of the same item).  Products of both side by side would end
    // together, and the softmax would wait for both.  The turn also says that the columns of tile
    // g - 2's scores are free for tile g's: the values waited for the first half's weights, and these
    // come behind the vote that every softmax thread of a CTA joins once its scores are loaded.
    // Without that vote the threads of the second half could still be loading.  A warp goes through
    // its loop together; one lane issues.
    constexpr uint32_t kFormat = H::kExponent == 0x7F80u ? 1u : 0u;  // bf16 or f16
    // fp32 accumulators, both operands of T, 128 rows; for P V the second has its dims outermost
    constexpr uint32_t kCommon = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (8u << 24);
    constexpr uint32_t kScores = kCommon | ((uint32_t)(kKeys / 8) << 17);
    constexpr uint32_t kValues = kCommon | (1u << 16) | (32u << 17);  // 256 dims, 128 a CTA
    const bool on = elect_one();
    uint32_t g = 0, slot = 0, phase = 0;
    bool ok = true;
    Walk cur = walk_from(p, sh.start, range, p.item_cost);
    if (warp == 10) {
      const uint64_t q_desc = operand_desc(q_at, 16, 1024), k_desc = operand_desc(k_at, 16, 1024);
      const uint64_t k_whole = operand_desc(k_at, 16, k_eight);
      uint32_t segments = 0;
      while (ok && cur.advance(p, kKeys)) {
        ok = wait_all(&sh.q_full, segments & 1u);
        for (int i = 0; i < cur.count && ok; ++i, ++g) {
          for (int x = 0; x < groups && ok; ++x) {
            ok = wait_all(&sh.k_full[slot], phase) &&
                 (x > 0 || g < 2 || wait_all(&sh.v_turn[g & 1u], (g >> 1) + 1u & 1u));
            if (!ok) break;
            tc_after_sync();
            const bool whole = x < whole_groups;
            uint64_t a = q_desc + x * (L::kKBytes / 16);
            uint64_t b = (whole ? k_whole : k_desc) + slot * (L::kKBytes / 16);
            const uint32_t step = (whole ? k_chunk : L::kChunkBytes) / 16;
            const int here = chunks - x * L::kGroup;
            bool add = x > 0;
#pragma unroll 1
            for (int c = min(here, L::kGroup); c > 0; --c) {  // zeros lie behind a row's end
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pair_mma(on, s_col(g), a + k * 2, b + k * 2, kScores, add || k > 0);
              add = true;
              a += L::kChunkBytes / 16;
              b += step;
            }
            pair_commit(on, &sh.k_empty[slot]);
            if (x == groups - 1) mbar_arrive(&sh.s_turn[g & 1u]);
            if (++slot == L::kKSlots) slot = 0, phase ^= 1u;
          }
          if (!ok) break;
          pair_commit(on, &sh.s_full[g & 1u]);
          if (i + 1 == cur.count) pair_commit(on, &sh.q_empty);
        }
        ++segments;
      }
    } else {
      const uint64_t p_desc = operand_desc(p_at, 16, 1024);
      // a piece of values, 16 positions after 16: within a run, or in the next ones
      const uint64_t v_desc = operand_desc(v_at, v_chunk, rows == 8 ? v_run : 1024u);
      while (ok && cur.advance(p, kKeys)) {
        for (int i = 0; i < cur.count && ok; ++i, ++g) {
#pragma unroll 1
          for (int s = 0; s < 2; ++s) {
            ok = ok && wait_all(&sh.v_full[slot], phase) &&
                 wait_all(&sh.p_full[s][g & 1u], (g >> 1) & 1u) &&
                 (s > 0 || i + 1 == cur.count ||
                  wait_all(&sh.s_turn[(g + 1) & 1u], ((g + 1) >> 1) & 1u));
            if (!ok) break;
            tc_after_sync();
            const uint64_t a = p_desc + s * (8192 / 16);
            const uint64_t b = v_desc + slot * (L::kVBytes / 16);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const uint32_t step = (16 * k >> shift) * v_run + (16 * k & (rows - 1)) * 128;
#pragma unroll
              for (int j = 0; j < DV / 256; ++j)
                pair_mma(on, o_col + j * 128, a + k * 2, b + step / 16 + j * (2 * v_chunk / 16),
                         kValues, i > 0 || s + k > 0);
            }
            pair_commit(on, &sh.v_empty[slot]);
            pair_commit(on, &sh.o_full[s]);
            // the other warp needs as long to see it as the rest takes
            if (s == 0) mbar_arrive(&sh.v_turn[g & 1u]);
            if (++slot == L::kVSlots) slot = 0, phase ^= 1u;
          }
        }
      }
    }
    // nothing is in flight when the tensor memory is given back
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q tcgen05.commit.cta_group::2"
        ".mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(&sh.drained)),
        "r"((uint32_t)on)
        : "memory");
    mbar_wait_bounded(&sh.drained, 0);
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  if (tid == 0) {
    pair_store(in_cta(smem_u32(&sh.peer_failed), rank ^ 1u), sh.failed);
    for (int i = 0; i < 3; ++i)
      pair_store(in_cta(smem_u32(&sh.peer_issued[i]), rank ^ 1u), sh.issued[i]);
  }
  __syncwarp();
  cluster_sync();
  tc_after_sync();
  const bool failed = sh.failed || sh.peer_failed;
  // After a wait that expired copies may be in flight.  CTA 0, whose barriers they complete on,
  // arrives in place of a CTA that did not come to a copy and waits for what the other one asked
  // for; without such a wait every copy has been multiplied.
  if (failed && rank == 0 && warp >= 8 && warp != 10) {
    const int of = warp == 11 ? 2 : warp - 8;
    const uint32_t slots = of == 0 ? L::kKSlots : of == 1 ? L::kVSlots : 1;
    uint64_t* full = of == 0 ? sh.k_full : of == 1 ? sh.v_full : &sh.q_full;
    const uint32_t a = sh.issued[of], b = sh.peer_issued[of];
    const uint32_t most = a > b ? a : b, least = a > b ? b : a;
    for (uint32_t n = most > slots ? most - slots : 0u; n < most; ++n) {
      if (n >= least && lane == 0) pair_arrive(in_cta(smem_u32(&full[n % slots]), 0));
      __syncwarp();
      mbar_wait_bounded(&full[n % slots], (n / slots) & 1u);
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp == 10)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  // The requests of the range are refused; what the pair has written of them may be unfinished:
  // NaN takes its place, and in the parts the joining kernel's sums.
  if (!failed) return;
  Walk cur = walk_from(p, sh.start, range, p.item_cost);
  Lost lost = {cur.b, -1};
  while (cur.advance(p, kKeys)) {
    lost.last = cur.b;
    const int64_t slot = cur.slot(pair) * p.part_rows;
    const int first = cur.head * 128 + (int)rank * 64;
    for (int r = tid; r < min(64, all_rows - first); r += kLatentThreads) {
      const int64_t to = (int64_t)cur.b * all_rows + first + r;
      const int part_row = (int)rank * 64 + r;
      if (!DSPARK_CHECK(cur.whole() ? row_held(p, to) : part_held(p, slot, part_row))) continue;
      if (!cur.whole()) {
        ws.stats[slot + part_row] = make_float2(NAN, NAN);
        continue;
      }
      for (int d = 0; d < p.latent; d += 2)
        *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + to * p.latent + d) =
            H::pack(NAN, NAN);
      if (p.lse) p.lse[to] = NAN;
    }
  }
  if (tid == 0 && rank == 0 && DSPARK_CHECK(pair < p.max_ctas)) ws.lost[pair] = lost;
}

// ------------------------------------------------------- the joining kernel
// The item that is first cut between pairs x and x + 1, if there is one, is
// joined from the pairs' partial rows, in the pairs' order: a warp takes 256
// dims of a row, four parts in flight together.  CTA (x, 0) also gives the
// requests that pair x lost their status.
constexpr int kLatentJoinThreads = 128;

template <typename T, int DV>
__global__ void __launch_bounds__(kLatentJoinThreads, 8)
    latent_join_kernel(const __grid_constant__ LatentParams p) {
  using H = Half<T>;
  constexpr int kSlices = DV / 256, kRows = kLatentJoinThreads / 32 / kSlices, kAhead = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Workspace ws = carve(p.workspace, p.part_rows, p.max_ctas);
  if (!DSPARK_CHECK(gridDim.x <= p.max_ctas)) return;
  const Seam at = ws.seam[min(blockIdx.x + 1, gridDim.x - 1)];
  Lost lost = {0, -1};
  if (blockIdx.y == 0 && threadIdx.x == 0) lost = ws.lost[blockIdx.x];
  [&] {
    const int c0 = blockIdx.x, c1 = blockIdx.x + 1 < gridDim.x ? at.last : -1;  // the item's pairs
    if (c1 < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * kRows + warp / kSlices, d = warp % kSlices * 256 + lane * 4;
    const int row = at.head * 128 + r, all_rows = p.nodes * p.heads;
    if (r >= p.part_rows || row >= all_rows) return;
    auto part_of = [&](int c) -> int64_t { return (2ll * c + (c == c0 ? 1 : 0)) * p.part_rows; };
    if (!DSPARK_CHECK(c1 < gridDim.x && part_held(p, part_of(c0), r) && part_held(p, part_of(c1), r)))
      return;
    const int64_t to = (int64_t)at.b * all_rows + row;
    if (!DSPARK_CHECK(row_held(p, to))) return;
    // kAhead parts of the row, beside the loads of what they are weighted with
    float4 x[kAhead], y[kAhead];
    auto load = [&](int c) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float4* v = reinterpret_cast<const float4*>(
            ws.rows + (part_of(min(c + u, c1)) + r) * DV + d);
        x[u] = __ldcs(v);
        y[u] = __ldcs(v + 32);
      }
    };
    load(c0);
    float2 st = make_float2(-INFINITY, 0.0f);  // of the lane's part
    if (c0 + lane <= c1) st = ws.stats[part_of(c0 + lane) + r];
    float top = st.x;
    for (int c = c0 + 32 + lane; c <= c1; c += 32) top = fmaxf(top, ws.stats[part_of(c) + r].x);
    top = warp_reduce(top, OpMaxF());
    const float safe = top == -INFINITY ? 0.0f : top;
    float f = exp2_approx(st.x - safe), all = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
    for (int c = c0; c <= c1; c += kAhead) {
      if (c > c0) load(c);
      if (c > c0 && (c - c0) % 32 == 0) {  // the next 32 parts, whose factors the lanes hold
        st = make_float2(-INFINITY, 0.0f);
        if (c + lane <= c1) st = ws.stats[part_of(c + lane) + r];
        f = exp2_approx(st.x - safe);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (c + u > c1) continue;
        const float w = __shfl_sync(0xffffffffu, f, (c + u - c0) & 31);
        all += __shfl_sync(0xffffffffu, st.y, (c + u - c0) & 31) * w;
        a = make_float4(a.x + x[u].x * w, a.y + x[u].y * w, a.z + x[u].z * w, a.w + x[u].w * w);
        b = make_float4(b.x + y[u].x * w, b.y + y[u].y * w, b.z + y[u].z * w, b.w + y[u].w * w);
      }
    }
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    T* out = static_cast<T*>(p.out) + to * p.latent + d;
    if (d < p.latent)
      *reinterpret_cast<uint2*>(out) =
          make_uint2(H::pack(a.x * inv, a.y * inv), H::pack(a.z * inv, a.w * inv));
    if (d + 128 < p.latent)
      *reinterpret_cast<uint2*>(out + 128) =
          make_uint2(H::pack(b.x * inv, b.y * inv), H::pack(b.z * inv, b.w * inv));
    if (d == 0 && p.lse)
      p.lse[to] = all == 0.0f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
  }();
  for (int b = lost.first; b <= lost.last; ++b) p.status[b] = DSPARK_ST_TIMEOUT;
}

}  // namespace attn
}  // namespace dspark
