// tree_attention.cu -- dspark_tree_attention: the nodes of a speculative step
// attend to their request's paged cache and to the nodes their tree shows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#define DSPARK_TU 12  // this file's number in the checked build's site codes
#include "common.cuh"

namespace dspark {

namespace {

struct AParams {
  const void* q;
  int64_t q_req, q_node, q_head;
  int B, nodes, heads, kv_heads;
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
  float scale;
  void* out;
  float* lse;
  int32_t* status;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

constexpr int kSimpleThreads = 128;

}  // namespace

// One CTA per (node, head, request); its warps take the positions in turn,
// each with a running maximum and sum, and are joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kSimpleThreads) tree_attention_simple_kernel(const AParams p) {
  constexpr int kPer = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % p.heads, t = blockIdx.x / p.heads, b = blockIdx.y;
  const int kvh = h / (p.heads / p.kv_heads);
  const int ctx = p.ctx[b], n = p.n_nodes[b];
  const bool bad = ctx < 0 || n < 0 || n > p.nodes ||
                   (int64_t)ctx + n > (int64_t)p.max_blocks * p.page;
  if (threadIdx.x == 0 && blockIdx.x == 0) p.status[b] = bad ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;
  const int64_t row = ((int64_t)b * p.nodes + t) * p.heads + h;

  float q[kPer], o[kPer];
  const T* qr = static_cast<const T*>(p.q) + b * p.q_req + t * p.q_node + h * p.q_head;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = bad || t >= n ? 0.0f : to_f32(qr[lane * kPer + i]) * p.scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int len = bad || t >= n ? 0 : ctx + n;
  const uint64_t seen = p.mask ? p.mask[(int64_t)b * p.nodes + t] : (2ull << t) - 1ull;
  for (int i = warp; i < len; i += 4) {
    if (i >= ctx && !((seen >> (i - ctx)) & 1ull)) continue;
    const int block = p.table[b * p.table_ld + i / p.page];
    if (block < 0 || block >= p.n_blocks) continue;
    const int64_t at = block * p.block_stride + (int64_t)(i % p.page) * p.token_stride +
                       kvh * p.head_stride + lane * kPer;
    const T* k = static_cast<const T*>(p.k) + at;
    const T* v = static_cast<const T*>(p.v) + at;
    float s = 0.0f;
#pragma unroll
    for (int d = 0; d < kPer; ++d) s = fmaf(q[d], to_f32(k[d]), s);
    s = warp_reduce(s, [](float a, float c) { return a + c; });
    const float top = fmaxf(m, s);
    const float safe = top == -INFINITY ? 0.0f : top;
    const float scale = expf(m - safe), w = expf(s - safe);
    m = top;
    l = l * scale + w;
#pragma unroll
    for (int d = 0; d < kPer; ++d) o[d] = o[d] * scale + w * to_f32(v[d]);
  }
#pragma unroll
  for (int d = 0; d < kPer; ++d) s_o[warp][lane * kPer + d] = o[d];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
  const float safe = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (int w = 0; w < 4; ++w) sum += s_l[w] * expf(s_m[w] - safe);
  for (int d = threadIdx.x; d < D; d += kSimpleThreads) {
    float a = 0.0f;
    for (int w = 0; w < 4; ++w) a += s_o[w][d] * expf(s_m[w] - safe);
    static_cast<T*>(p.out)[row * D + d] = from_f32<T>(sum > 0.0f ? a / sum : (sum == 0.0f ? 0.0f : a / sum));
  }
  if (threadIdx.x == 0 && p.lse) p.lse[row] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

int64_t tree_attention_workspace_bytes(int B, int nodes, int heads, int kv_heads, int head_dim) {
  return 16;
}

template <typename T>
static void launch_simple(const AParams& p, int head_dim, dim3 grid, cudaStream_t stream) {
  if (head_dim == 64)
    tree_attention_simple_kernel<T, 64><<<grid, kSimpleThreads, 0, stream>>>(p);
  else if (head_dim == 128)
    tree_attention_simple_kernel<T, 128><<<grid, kSimpleThreads, 0, stream>>>(p);
  else
    tree_attention_simple_kernel<T, 256><<<grid, kSimpleThreads, 0, stream>>>(p);
}

cudaError_t launch_tree_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                  int64_t q_head, int B, int nodes, int heads, int kv_heads,
                                  int head_dim, const void* k, const void* v,
                                  int64_t block_stride, int64_t token_stride, int64_t head_stride,
                                  int n_blocks, int page, const int32_t* table, int64_t table_ld,
                                  int max_blocks, const int32_t* ctx, const int32_t* n_nodes,
                                  const uint64_t* mask, float scale, void* out, float* lse,
                                  int32_t* status, void* workspace, cudaStream_t stream) {
  AParams p;
  p.q = q;
  p.q_req = q_req;
  p.q_node = q_node;
  p.q_head = q_head;
  p.B = B;
  p.nodes = nodes;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.k = k;
  p.v = v;
  p.block_stride = block_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.n_blocks = n_blocks;
  p.page = page;
  p.table = table;
  p.table_ld = table_ld;
  p.max_blocks = max_blocks;
  p.ctx = ctx;
  p.n_nodes = n_nodes;
  p.mask = mask;
  p.scale = scale;
  p.out = out;
  p.lse = lse;
  p.status = status;
  const dim3 grid((unsigned)(nodes * heads), (unsigned)B);
  if (dtype == DSPARK_BF16)
    launch_simple<__nv_bfloat16>(p, head_dim, grid, stream);
  else
    launch_simple<__half>(p, head_dim, grid, stream);
  return cudaGetLastError();
}

DSPARK_CHECK_COLLECTOR(tree_attention)

}  // namespace dspark
