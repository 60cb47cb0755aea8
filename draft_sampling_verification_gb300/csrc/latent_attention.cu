// latent_attention.cu -- dspark_latent_attention: the nodes of a speculative
// step attend to their request's latent cache, whose rows are the keys and,
// in their first elements, the values of every head.  Host side; the kernels
// are in latent_attention.cuh.
#define DSPARK_TU 16  // this file's number in the checked build's site codes

#include "latent_attention.cuh"

namespace dspark {
namespace attn {
namespace {

constexpr int kMaxPairs = 80;  // 160 SMs at most are used

int values_dim(int latent) { return latent <= 256 ? 256 : 512; }  // of the kernel
int latent_part_rows(int rows) { return rows >= 128 ? 128 : (rows + 7) / 8 * 8; }

template <typename T>
bool map_rows(CUtensorMap* map, const LatentParams& p, int rows) {
  const auto encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t sizes[3] = {(cuuint64_t)p.width, (cuuint64_t)p.page, (cuuint64_t)p.n_blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.block_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  return encode(map,
                Half<T>::kExponent == 0x7F80u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                3, const_cast<void*>(p.k), sizes, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DV>
cudaError_t launch(const LatentParams& p, int sms, cudaStream_t stream) {
  using L = Latent<DV>;
  const int rows = wide_box_rows(p.page, 64);
  CUtensorMap map;
  if (!map_rows<T>(&map, p, rows)) return cudaErrorInvalidValue;
  auto* kernel = latent_attention_kernel<T, DV>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const int pairs = min(kMaxPairs, max(1, sms / 2));
  kernel<<<2 * pairs, kLatentThreads, L::kSmem, stream>>>(p, map, rows);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while that one runs, waits on the device for its end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs, (p.part_rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_join_kernel<T, DV>, p);
}

}  // namespace

DSPARK_STALL_SETTER(latent)

}  // namespace attn

int64_t latent_attention_workspace_bytes(int B, int nodes, int heads, int latent) {
  return attn::workspace_bytes(attn::latent_part_rows(nodes * heads), attn::values_dim(latent),
                               attn::kMaxPairs);
}

cudaError_t launch_latent_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                    int64_t q_head, int B, int nodes, int heads, int latent,
                                    int rope, const void* cache, int64_t block_stride,
                                    int64_t token_stride, int n_blocks, int page,
                                    const int32_t* table, int64_t table_ld, int max_blocks,
                                    const int32_t* ctx, const int32_t* n_nodes,
                                    const uint64_t* mask, float scale, void* out, float* lse,
                                    int32_t* status, void* workspace, cudaStream_t stream) {
  attn::LatentParams p;
  p.q = q;
  p.q_req = q_req;
  p.q_node = q_node;
  p.q_head = q_head;
  p.B = B;
  p.nodes = nodes;
  p.heads = heads;
  p.kv_heads = (nodes * heads + 127) / 128;  // an item for each 128 rows of a request
  p.group = heads;
  p.k = p.v = cache;
  p.block_stride = block_stride;
  p.token_stride = token_stride;
  p.head_stride = 0;
  p.n_blocks = n_blocks;
  p.page = page;
  p.table = table;
  p.table_ld = table_ld;
  p.max_blocks = max_blocks;
  p.ctx = ctx;
  p.n_nodes = n_nodes;
  p.mask = mask;
  p.scale2 = scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.workspace = static_cast<char*>(workspace);
  p.max_ctas = attn::kMaxPairs;
  p.tile = attn::kLatentKeys;
  p.item_cost = attn::kLatentCost;
  p.row_tiles = 1;
  p.part_rows = attn::latent_part_rows(nodes * heads);
  p.part_wide = 8;
  p.waits = true;
  p.latent = latent;
  p.width = latent + rope;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool wide = attn::values_dim(latent) == 512;
  if (dtype == DSPARK_BF16)
    return wide ? attn::launch<__nv_bfloat16, 512>(p, sms, stream)
                : attn::launch<__nv_bfloat16, 256>(p, sms, stream);
  return wide ? attn::launch<__half, 512>(p, sms, stream)
              : attn::launch<__half, 256>(p, sms, stream);
}

DSPARK_CHECK_COLLECTOR(latent_attention)

}  // namespace dspark
