// latent_attention.cu -- dspark_latent_attention: the nodes of a speculative
// step attend to their request's latent cache, whose rows are the keys and,
// in their first elements, the values of every head.
#define DSPARK_TU 16  // this file's number in the checked build's site codes

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPairs = (DSPARK_MAX_LATENT + DSPARK_MAX_LATENT_ROPE) / 64;  // of a lane

struct Params {
  const void* q;
  int64_t q_req, q_node, q_head;
  int B, nodes, heads, latent, width;
  const void* cache;
  int64_t block_stride, token_stride;
  int n_blocks, page;
  const int32_t* table;
  int64_t table_ld;
  int max_blocks;
  const int32_t* ctx;
  const int32_t* n_nodes;
  const uint64_t* mask;
  float scale;
  void* out;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float2 widen(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 widen(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ void narrow(float2 v, __nv_bfloat162* to) {
  *to = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void narrow(float2 v, __half2* to) {
  *to = __floats2half2_rn(v.x, v.y);
}

// A CTA per row (request, node, head), a warp per position, the warps'
// softmax states joined at the end.
template <typename T2>
__global__ void __launch_bounds__(kThreads) latent_attention_kernel(const Params p) {
  __shared__ float s_max[kWarps], s_sum[kWarps], s_out[DSPARK_MAX_LATENT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, node = blockIdx.x / p.heads, head = blockIdx.x % p.heads;
  int ctx = p.ctx[b], n = p.n_nodes[b];
  const bool bad =
      ctx < 0 || n < 0 || n > p.nodes || (int64_t)ctx + n > (int64_t)p.max_blocks * p.page;
  if (bad) ctx = n = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.status[b] = bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;
  uint64_t mask = 0;
  if (node < n) mask = p.mask ? p.mask[(int64_t)b * p.nodes + node] : ~0ull >> (63 - node);
  const T2* q = reinterpret_cast<const T2*>(static_cast<const char*>(p.q) +
                                            2 * (b * p.q_req + node * p.q_node + head * p.q_head));
  float2 x[kPairs], a[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int d = i * 64 + lane * 2;
    x[i] = d < p.width ? widen(q[d / 2]) : make_float2(0.0f, 0.0f);
    a[i] = make_float2(0.0f, 0.0f);
  }
  float top = -INFINITY, sum = 0.0f;
  const int len = node < n ? ctx + n : 0;
  for (int i = warp; i < len; i += kWarps) {
    if (i >= ctx && !((mask >> (i - ctx)) & 1)) continue;
    const int block = p.table[b * p.table_ld + i / p.page];
    if (block < 0 || block >= p.n_blocks) continue;
    const T2* row = reinterpret_cast<const T2*>(
        static_cast<const char*>(p.cache) +
        2 * (block * p.block_stride + (int64_t)(i % p.page) * p.token_stride));
    float2 k[kPairs];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int d = j * 64 + lane * 2;
      if (d >= p.width) continue;
      k[j] = widen(row[d / 2]);
      s += x[j].x * k[j].x + x[j].y * k[j].y;
    }
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    s *= p.scale;
    const float m = fmaxf(top, s), f = top == m ? 1.0f : expf(top - m);
    const float e = m == -INFINITY ? 0.0f : expf(s - m);
    top = m;
    sum = sum * f + e;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (j * 64 >= p.latent) continue;
      a[j].x = a[j].x * f + e * k[j].x;
      a[j].y = a[j].y * f + e * k[j].y;
    }
  }
  if (lane == 0) {
    s_max[warp] = top;
    s_sum[warp] = sum;
  }
  __syncthreads();
  float all = -INFINITY, total = 0.0f;
  for (int w = 0; w < kWarps; ++w) all = fmaxf(all, s_max[w]);
  const float safe = all == -INFINITY ? 0.0f : all;
  for (int w = 0; w < kWarps; ++w) total += s_sum[w] * expf(s_max[w] - safe);
  const float f = total == 0.0f ? 0.0f : expf(top - safe) / total;
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const int d = j * 64 + lane * 2;
        if (d >= p.latent) continue;
        s_out[d] = (w ? s_out[d] : 0.0f) + a[j].x * f;
        s_out[d + 1] = (w ? s_out[d + 1] : 0.0f) + a[j].y * f;
      }
    }
    __syncthreads();
  }
  const int64_t to = ((int64_t)b * p.nodes + node) * p.heads + head;
  T2* out = static_cast<T2*>(p.out) + to * (p.latent / 2);
  for (int d = threadIdx.x; d < p.latent / 2; d += kThreads)
    narrow(make_float2(s_out[2 * d], s_out[2 * d + 1]), &out[d]);
  if (threadIdx.x == 0 && p.lse) p.lse[to] = total == 0.0f ? -INFINITY : all + logf(total);
}

}  // namespace

int64_t latent_attention_workspace_bytes(int B, int nodes, int heads, int latent) { return 16; }

cudaError_t launch_latent_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                    int64_t q_head, int B, int nodes, int heads, int latent,
                                    int rope, const void* cache, int64_t block_stride,
                                    int64_t token_stride, int n_blocks, int page,
                                    const int32_t* table, int64_t table_ld, int max_blocks,
                                    const int32_t* ctx, const int32_t* n_nodes,
                                    const uint64_t* mask, float scale, void* out, float* lse,
                                    int32_t* status, void* workspace, cudaStream_t stream) {
  const Params p = {q,          q_req,   q_node, q_head,       B,            nodes,  heads,
                    latent,     latent + rope,   cache,        block_stride, token_stride,
                    n_blocks,   page,    table,  table_ld,     max_blocks,   ctx,    n_nodes,
                    mask,       scale,   out,    lse,          status};
  const dim3 grid(nodes * heads, B);
  if (dtype == DSPARK_BF16)
    latent_attention_kernel<__nv_bfloat162><<<grid, kThreads, 0, stream>>>(p);
  else
    latent_attention_kernel<__half2><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

DSPARK_CHECK_COLLECTOR(latent_attention)

}  // namespace dspark
