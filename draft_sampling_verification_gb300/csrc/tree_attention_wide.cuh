// tree_attention_wide.cuh -- the attention kernel for items of more than 64
// rows (wide trees, many query heads to a cached head), on the fifth
// generation's tensor instructions.  Included by the translation units of
// tree_attention.cuh.
#pragma once

#include <cuda.h>

#include "tree_attention.cuh"

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
// one box of a cache, from (dim x, row r of head h of block b), completing on `bar`; a block
// beyond the cache gives zeros
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, int x, int r,
                                             int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(r), "r"(h), "r"(b), "r"(smem_u32(bar))
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
// Up to 256 rows of an item, as two tiles of 128, over tiles of 128
// positions: S = Q K^T into tensor memory, softmax by the warpgroup that owns
// the row tile (a thread per row, so no exchange between threads), the
// weights back into tensor memory over the scores, O += P V.  The two row
// tiles alternate: the tensor cores work for one while the other is in its
// softmax.  Bound by the products (2 * 2 * 128 * 128 * D operations per row
// tile and step) and, beside them, the exponentials.
//
// The products run in the order they are issued, so the barrier of a tile's
// scores also says that its accumulators hold every earlier step: the
// softmax warpgroup may then rescale them.  It does so only when a score
// passes the row's reference by more than 8, as in the streaming kernel.
//
// Warps 0-3 and 4-7: softmax, Q and the results of row tile 0 and 1.  Warp 8:
// tensor copies of keys and values, box by box of a block's rows, into a ring
// of stages each.  Warp 9: issues the products.  Warps 10-11: where a tile
// holds nodes, clear its values of infinities and NaN.  K and Q lie in rows
// of 64 dims (128 bytes, swizzled in groups of eight rows); V the same, read
// with dims as its major axis.
constexpr int kWideThreads = 384;  // 168 registers a thread: a row's 128 scores and more
constexpr int kWideTile = 128;

template <int D>
struct Wide {
  static constexpr int kHalves = D / 64;
  static constexpr int kOperand = 128 * D * 2;  // bytes of 128 rows of Q, K or V
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kSmem = (2 + 2 * kStages) * kOperand + 1024;
};
constexpr int kWideMaxStages = 4;
constexpr int kClearThreads = 64;

struct WideShared {
  uint64_t k_full[kWideMaxStages], k_empty[kWideMaxStages];
  uint64_t v_full[kWideMaxStages], v_empty[kWideMaxStages];
  uint64_t v_nodes[kWideMaxStages], v_clear[kWideMaxStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drained;
  uint64_t scan[32];
  Start start;
  uint32_t valid[8][4];  // a tile's positions that hold a key, by tile number modulo 8
  uint32_t special[8];   // a value of a tile's nodes is an infinity or a NaN
  uint32_t tmem;
  uint32_t failed;       // a wait expired
};

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads, 1)
    tree_attention_wide_kernel(const __grid_constant__ Params p,
                               const __grid_constant__ CUtensorMap k_map,
                               const __grid_constant__ CUtensorMap v_map, int box_rows) {
  using H = Half<T>;
  using W = Wide<D>;
  constexpr int kChunks = D / 8, kStages = W::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ WideShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, k_at = base + 2 * W::kOperand, v_at = k_at + kStages * W::kOperand;

  const Workspace ws = carve(p.workspace, kWideRows);
  const int64_t range = find_range<kWideThreads>(p, kWideTile, ws, sh.scan, &sh.start);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (range <= 0) return;
  Walk cur = walk_from(sh.start, range);
  const int r0 = (blockIdx.x % p.row_tiles) * kWideRows;
  const int n_tiles = p.nodes * p.group - r0 > 128 ? 2 : 1;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.v_nodes[i], 1);
      mbar_init(&sh.v_clear[i], kClearThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 128);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.o_full[i], 1);
    }
    mbar_init(&sh.drained, 1);
    sh.failed = 0u;
    mbar_init_fence();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  // columns: the scores of row tile m (the weights over their first half), then its accumulators
  const uint32_t tmem = sh.tmem;
  auto s_col = [&](int m) -> uint32_t { return tmem + 128u * m; };
  auto o_col = [&](int m) -> uint32_t { return tmem + 256u + 128u * m; };

  // a bounded wait; once one expires, every later one of the CTA gives up at once
  auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    if (mbar_try_wait(bar, phase)) return true;
    if (*(volatile uint32_t*)&sh.failed) return false;
    if (mbar_wait_bounded(bar, phase)) return true;
    *(volatile uint32_t*)&sh.failed = 1u;
    return false;
  };
  if (warp < 8) {
    // -------------------------------------------------- softmax and results
    const int m = warp >> 2;
    const int t = tid & 127;  // this thread's row of the tile and lane of tensor memory
    const uint32_t sc = s_col(m) + ((uint32_t)(t & ~31) << 16);
    const uint32_t oc = o_col(m) + ((uint32_t)(t & ~31) << 16);
    // a negative scale goes into Q's sign, so that the largest score stays the largest; 0 would
    // make NaN of a hidden score
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;
    const float scale = fmaxf(fabsf(p.scale2), 1.17549435e-38f);
    uint32_t tile_no = 0, segments = 0;
    bool ok = m < n_tiles;
    // the item's Q: 16-byte pieces of this thread's column, every kStep-th row
    constexpr int kStep = 128 / kChunks;
    uint4 q[kChunks];
    auto load_q = [&](const Walk& w) {
      const int live = request_lengths(p, w.b).nodes * p.group;
      const T* from = static_cast<const T*>(p.q) + w.b * p.q_req + (t % kChunks) * 8;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int row = r0 + m * 128 + i * kStep + t / kChunks;
        const int at = row < live ? row : 0, node = at / p.group;  // no branch: all loads at once
        const int h = w.head * p.group + at - node * p.group;
        const T* piece = from + node * p.q_node + h * p.q_head;
        q[i] = live > 0 ? __ldg(reinterpret_cast<const uint4*>(piece)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t keep = row < live ? ~0u : 0u;
        q[i] = make_uint4((q[i].x ^ flip) & keep, (q[i].y ^ flip) & keep, (q[i].z ^ flip) & keep,
                          (q[i].w ^ flip) & keep);
      }
    };
    auto store_q = [&] {
      const int c = t % kChunks;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int r = i * kStep + t / kChunks;
        const uint32_t to = q_at + m * W::kOperand + (c >> 3) * 16384 + r * 128 +
                            (((c & 7) ^ (r & 7)) << 4);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(q[i].x),
                     "r"(q[i].y), "r"(q[i].z), "r"(q[i].w)
                     : "memory");
      }
      fence_async_shared();
      mbar_arrive(&sh.q_full[m]);
    };
    bool more = ok && cur.advance(p, kWideTile);
    if (more) {
      load_q(cur);
      store_q();
    }
    while (ok && more) {
      const int tiles = cur.count;
      const Lengths len = request_lengths(p, cur.b);
      const int live = len.nodes * p.group;
      if (tid == 0 && r0 == 0 && cur.head == 0 && cur.first == 0)
        p.status[cur.b] = len.bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;

      const int row = r0 + m * 128 + t, node = row / p.group;
      uint64_t mask = 0;
      if (row < live)
        mask = p.mask ? p.mask[(int64_t)cur.b * p.nodes + node] : ~0ull >> (63 - node);
      float ref = -INFINITY;
      float2 sum2 = make_float2(0.0f, 0.0f);
      bool special = false;
      for (int i = 0; i < tiles; ++i, ++tile_no) {
        ok = __all_sync(0xffffffffu, wait(&sh.s_full[m], tile_no & 1u));
        if (!ok) break;
        tc_after_sync();
        if (i > 0) special |= sh.special[(tile_no - 1u) & 7u] != 0u;
        const int pos = (cur.first + i) * kWideTile;
        const uint32_t* words = sh.valid[tile_no & 7u];
        const bool plain = pos + kWideTile <= len.ctx &&
                           (words[0] & words[1] & words[2] & words[3]) == 0xFFFFFFFFu;
        float v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32(v + c * 32, sc + c * 32);
        tmem_wait_load();
        if (!plain) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w = words[c];
            const int node0 = pos + c * 32 - len.ctx;  // the node of the chunk's first position
            if (node0 >= 0)
              w &= node0 < 64 ? (uint32_t)(mask >> node0) : 0u;
            else if (node0 > -32)
              w &= (uint32_t)(mask << -node0) | ((1u << -node0) - 1u);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((w >> j) & 1u)) v[c * 32 + j] = -INFINITY;
          }
        }
        float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 124; j += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(fmaxf(m4[k], v[j + k]), v[j + 4 + k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], v[124 + k]);
        float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
          top = fmaxf(top, ref);
          const float f = top == -INFINITY ? 1.0f : exp2_approx(ref - top);
          ref = top;
          sum2.x *= f;
          sum2.y *= f;
          if (i > 0) {
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
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 x = fma2_rn(make_float2(v[c * 32 + 2 * j], v[c * 32 + 2 * j + 1]), by, off);
            x.x = exp2_approx(x.x);
            x.y = exp2_approx(x.y);
            if (j & 1)
              part2 = add2_rn(part2, x);
            else
              sum2 = add2_rn(sum2, x);
            w[j] = H::pack(x.x, x.y);
          }
          tmem_store16(sc + c * 16, w);
        }
        sum2 = add2_rn(sum2, part2);
        tmem_wait_store();
        tc_before_sync();
        mbar_arrive(&sh.p_full[m]);
      }
      // the next item's Q is on its way while this one's last products run, and
      // its first scores are computed while this one's results are written
      Walk ahead = cur;
      more = ok && ahead.advance(p, kWideTile);
      if (more) load_q(ahead);
      if (ok) ok = __all_sync(0xffffffffu, wait(&sh.o_full[m], segments & 1u));
      ++segments;
      if (!ok) break;
      tc_after_sync();
      if (more) store_q();
      special |= sh.special[(tile_no - 1u) & 7u] != 0u;

      float sum = sum2.x + sum2.y;
      if (row >= live) {  // a row of no node: its zero query saw the text all the same
        ref = -INFINITY;
        sum = 0.0f;
      }
      const bool full = cur.whole();
      const int h = cur.head * p.group + row - node * p.group;
      const int64_t to = ((int64_t)cur.b * p.nodes + node) * p.heads + h;
      const int64_t slot = cur.slot();
      const bool mine = row < p.nodes * p.group;
      const float inv = sum == 0.0f ? 0.0f : full ? 1.0f / sum : 1.0f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
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
            const int at = len.ctx + k, tile = at / kWideTile;
            if (!((mask >> k) & 1ull) || tile < cur.first || tile >= cur.first + tiles) continue;
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
        if (mine && full) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to * D + c * 32);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            out[j] = make_uint4(H::pack(v[8 * j] * inv, v[8 * j + 1] * inv),
                                H::pack(v[8 * j + 2] * inv, v[8 * j + 3] * inv),
                                H::pack(v[8 * j + 4] * inv, v[8 * j + 5] * inv),
                                H::pack(v[8 * j + 6] * inv, v[8 * j + 7] * inv));
        } else if (mine) {
          // whole 32-byte sectors: a warp's rows lie far apart
          float* out = ws.rows + (slot * kWideRows + m * 128 + t) * D + c * 32;
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + j),
                         "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3]), "f"(v[j + 4]),
                         "f"(v[j + 5]), "f"(v[j + 6]), "f"(v[j + 7])
                         : "memory");
        }
        __syncwarp();
      }
      if (mine) {
        if (!full)
          ws.stats[slot * kWideRows + m * 128 + t] = make_float2(ref, sum);
        else if (p.lse)
          p.lse[to] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      }
      tc_before_sync();  // the accumulators are read: the next item may take them
      cur = ahead;
    }
  } else if (warp != 9) {
    // ------------------------------------------------------ keys and values
    // Lane i copies the tile's box i, box_rows positions of one block.
    const int boxes = kWideTile / box_rows;  // at most 16
    uint32_t g = 0, turns = 0;  // turns: each stage's phase of the tiles with nodes
    bool ok = true;
    while (ok && cur.advance(p, kWideTile)) {
      const int tiles = cur.count;
      const Lengths len = request_lengths(p, cur.b);
      const int first = cur.first * kWideTile;
      if (warp == 8) {
        const int32_t* table = p.table + cur.b * p.table_ld;
        auto entry_of = [&](int i) -> int {
          const int pos = first + i * kWideTile + lane * box_rows;
          return i < tiles && lane < boxes && pos < len.len ? __ldg(table + pos / p.page) : -1;
        };
        int ahead = entry_of(0);
        for (int i = 0; i < tiles; ++i, ++g) {
          const int pos0 = first + i * kWideTile, pos = pos0 + lane * box_rows, block = ahead;
          ahead = entry_of(i + 1);
          const bool held = block >= 0 && block < p.n_blocks;
          const int from = held ? block : p.n_blocks, row = held ? pos % p.page : 0;
          const uint32_t held_boxes = __ballot_sync(0xffffffffu, held);
          const uint32_t stage = g % kStages, phase = (g / kStages) & 1u;
          ok = __all_sync(0xffffffffu, wait(&sh.k_empty[stage], phase ^ 1u));
          if (!ok) break;
          if (lane < 4) {
            uint32_t word = 0u;  // positions 32 lane .. of the tile
            if (box_rows >= 32) {
              word = (held_boxes >> (lane * 32 / box_rows)) & 1u ? ~0u : 0u;
            } else {
              for (int j = 0; j < 32 / box_rows; ++j)
                if ((held_boxes >> (lane * 32 / box_rows + j)) & 1u)
                  word |= ((1u << box_rows) - 1u) << (j * box_rows);
            }
            const int past = len.len - (pos0 + lane * 32);  // positions before the end
            sh.valid[g & 7u][lane] = past >= 32 ? word : past > 0 ? word & ((1u << past) - 1u) : 0u;
            sh.special[g & 7u] = 0u;
          }
          auto copy = [&](const CUtensorMap* map, uint32_t at, uint64_t* full) {
            if (lane == 0) mbar_arrive_expect_tx(full, W::kOperand);
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
              for (int h = 0; h < W::kHalves; ++h)
                tma_load_box(at + stage * W::kOperand + h * 16384 + lane * box_rows * 128, map,
                             h * 64, row, cur.head, from, full);
            }
          };
          copy(&k_map, k_at, &sh.k_full[stage]);
          ok = __all_sync(0xffffffffu, wait(&sh.v_empty[stage], phase ^ 1u));
          if (!ok) break;
          // values that are to be cleared first land on a barrier of their own
          const bool nodes_here = pos0 + kWideTile > len.ctx;
          copy(&v_map, v_at, nodes_here ? &sh.v_nodes[stage] : &sh.v_full[stage]);
          if (nodes_here && lane == 0) mbar_arrive(&sh.v_full[stage]);
        }
      } else {
        // Rows from the first node on: nodes, which some rows see and others
        // do not, and what lies behind the end.  0 times an infinity or a NaN
        // would reach rows that do not see it.
        for (int i = 0; i < tiles; ++i, ++g) {
          const int pos0 = first + i * kWideTile;
          if (pos0 + kWideTile <= len.ctx) continue;
          const uint32_t stage = g % kStages;
          ok = __all_sync(0xffffffffu, wait(&sh.v_nodes[stage], (turns >> stage) & 1u));
          if (!ok) break;
          turns ^= 1u << stage;
          const int from = max(0, len.ctx - pos0);
          for (int j = tid - 320; j < (kWideTile - from) * kChunks; j += kClearThreads) {
            const int r = from + j / kChunks, c = j % kChunks;
            const uint32_t addr = v_at + stage * W::kOperand + (c >> 3) * 16384 + r * 128 +
                                  (((c & 7) ^ (r & 7)) << 4);
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(addr)
                         : "memory");
            if (any_special<T>(w[0]) || any_special<T>(w[1]) || any_special<T>(w[2]) ||
                any_special<T>(w[3])) {
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                           "r"(without_special<T>(w[0])), "r"(without_special<T>(w[1])),
                           "r"(without_special<T>(w[2])), "r"(without_special<T>(w[3]))
                           : "memory");
              if (pos0 + r < len.len) *(volatile uint32_t*)&sh.special[g & 7u] = 1u;
            }
          }
          fence_async_shared();
          mbar_arrive(&sh.v_clear[stage]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------- products
    // The warp goes through the loop together; one lane issues.
    constexpr uint32_t kFormat = H::kExponent == 0x7F80u ? 1u : 0u;  // bf16 or f16
    // fp32 accumulators, both operands of T, 128 rows; for P V the second has its dims outermost
    constexpr uint32_t kCommon = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (8u << 24);
    constexpr uint32_t kScores = kCommon | ((kWideTile / 8u) << 17);
    constexpr uint32_t kValues = kCommon | (1u << 16) | (((uint32_t)D / 8u) << 17);
    const bool on = elect_one();
    // descriptors of Q's tiles, and of the stages of keys and values; an
    // operand further on adds its distance / 16
    const uint64_t q_desc = operand_desc(q_at, 16, 1024), k_desc = operand_desc(k_at, 16, 1024);
    const uint64_t v_desc = operand_desc(v_at, 16384, 1024);
    auto scores = [&](int m, uint32_t g) {
      const uint64_t a = q_desc + (uint32_t)m * (W::kOperand / 16);
      const uint64_t b = k_desc + (g % kStages) * (W::kOperand / 16);
#pragma unroll
      for (int kt = 0; kt < D / 16; ++kt) {
        constexpr int kHalf = 16384 / 16, kStep = 32 / 16;
        const uint32_t at = (kt >> 2) * kHalf + (kt & 3) * kStep;
        mma_ss(on, s_col(m), a + at, b + at, kScores, kt > 0);
      }
      mma_commit(on, &sh.s_full[m]);
    };
    auto values = [&](int m, uint32_t g, bool add) {
      const uint64_t b = v_desc + (g % kStages) * (W::kOperand / 16);
#pragma unroll
      for (int kt = 0; kt < kWideTile / 16; ++kt)
        mma_ts(on, o_col(m), s_col(m) + kt * 8, b + kt * (2048 / 16), kValues, add || kt > 0);
    };
    auto wait_all = [&](uint64_t* bar, uint32_t phase) -> bool {
      return __all_sync(0xffffffffu, wait(bar, phase));
    };
    auto phase_of = [](uint32_t g) -> uint32_t { return (g / kStages) & 1u; };
    uint32_t g = 0, segments = 0, turns = 0;
    bool ok = true;
    while (ok && cur.advance(p, kWideTile)) {
      const int tiles = cur.count;
      const Lengths len = request_lengths(p, cur.b);
      for (int m = 0; m < n_tiles; ++m) ok = ok && wait_all(&sh.q_full[m], segments & 1u);
      ok = ok && wait_all(&sh.k_full[g % kStages], phase_of(g));
      if (!ok) break;
      tc_after_sync();
      for (int m = 0; m < n_tiles; ++m) scores(m, g);
      mma_commit(on, &sh.k_empty[g % kStages]);
      for (int i = 0; i < tiles && ok; ++i, ++g) {
        const bool more = i + 1 < tiles;
        for (int m = 0; m < n_tiles; ++m) {
          ok = wait_all(&sh.p_full[m], g & 1u);
          if (m == 0) {
            ok = ok && wait_all(&sh.v_full[g % kStages], phase_of(g));
            if ((cur.first + i + 1) * kWideTile > len.ctx) {
              ok = ok && wait_all(&sh.v_clear[g % kStages], (turns >> (g % kStages)) & 1u);
              turns ^= 1u << (g % kStages);
            }
          }
          if (!ok) break;
          tc_after_sync();
          values(m, g, i > 0);
          if (m == n_tiles - 1) mma_commit(on, &sh.v_empty[g % kStages]);
          if (more) {
            if (m == 0) ok = wait_all(&sh.k_full[(g + 1u) % kStages], phase_of(g + 1u));
            if (!ok) break;
            scores(m, g + 1u);
          } else {
            mma_commit(on, &sh.o_full[m]);
          }
        }
        if (ok && more) mma_commit(on, &sh.k_empty[(g + 1u) % kStages]);
      }
      ++segments;
    }
    // nothing of this CTA's is in flight when its memory is given back
    mma_commit(on, &sh.drained);
    mbar_wait_bounded(&sh.drained, 0);
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  if (sh.failed && tid == 0) {  // the requests of this range are refused
    for (cur = walk_from(sh.start, range); cur.advance(p, kWideTile);)
      p.status[cur.b] = DSPARK_ST_TIMEOUT;
  }
}

// rows of a tensor copy: the most that divide a block and a tile; the swizzle
// wants whole groups of eight
inline int wide_box_rows(int page) {
  int rows = kWideTile;
  while (page % rows) rows /= 2;
  return rows;
}

// the map of one cache: dims, rows of a block, heads, blocks
template <typename T>
bool map_cache(CUtensorMap* map, const Params& p, const void* cache, int dim, int box_rows) {
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
  const cuuint64_t sizes[4] = {(cuuint64_t)dim, (cuuint64_t)p.page, (cuuint64_t)p.kv_heads,
                               (cuuint64_t)p.n_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.head_stride * 2,
                                 (cuuint64_t)p.block_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, steps[4] = {1, 1, 1, 1};
  return encode(map,
                Half<T>::kExponent == 0x7F80u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                4, const_cast<void*>(cache), sizes, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// false: the cache's shape has no map, or blocks too short for one
template <typename T, int D>
bool launch_wide(Params p, int sms, cudaStream_t stream, cudaError_t* error) {
  const int box_rows = wide_box_rows(p.page);
  CUtensorMap k_map, v_map;
  if (box_rows < 8 || !map_cache<T>(&k_map, p, p.k, D, box_rows) ||
      !map_cache<T>(&v_map, p, p.v, D, box_rows))
    return false;
  p.row_tiles = (p.nodes * p.group + kWideRows - 1) / kWideRows;
  auto* kernel = tree_attention_wide_kernel<T, D>;
  *error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Wide<D>::kSmem);
  if (*error != cudaSuccess) return true;
  const int grid = min(kMaxCtas, max(sms, p.row_tiles));
  kernel<<<grid, kWideThreads, Wide<D>::kSmem, stream>>>(p, k_map, v_map, box_rows);
  *error = cudaGetLastError();
  if (*error == cudaSuccess) *error = launch_join<T, D, 4>(p, kWideRows, grid, stream);
  return true;
}

template <typename T, int D>
cudaError_t launch_dim(const Params& p, int sms, cudaStream_t stream) {
  const int rows = shape_rows(p.nodes * p.group, D);
  if (rows == 8) return launch_shape<T, D, 1, 1>(p, sms, stream);
  if (rows == 16) return launch_shape<T, D, 2, 1>(p, sms, stream);
  if constexpr (D == 256) {
    if (rows == 32) return launch_shape<T, D, 2, 2>(p, sms, stream);
    return launch_shape<T, D, 2, 4>(p, sms, stream);
  } else {
    if (rows == 24) return launch_shape<T, D, 3, 1>(p, sms, stream);
    if (rows == 32) return launch_shape<T, D, 4, 1>(p, sms, stream);
    if (rows == 48) return launch_shape<T, D, 3, 2>(p, sms, stream);
    cudaError_t e;
    if (p.nodes * p.group > 64 && launch_wide<T, D>(p, sms, stream, &e)) return e;
    return launch_shape<T, D, 4, 2>(p, sms, stream);
  }
}

}  // namespace attn
}  // namespace dspark
