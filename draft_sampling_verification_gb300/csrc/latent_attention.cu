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

// Dims of the kernel's values.  64 requests of 4,000 tokens with 256 + 64 elements and 96 rows take
// 49 us in the kernel of 256 and 58 in that of 512.
int values_dim(int latent) { return latent <= 256 ? 256 : 512; }
int latent_part_rows(int rows) { return rows >= 128 ? 128 : (rows + 7) / 8 * 8; }

// a map of 16-bit elements; the innermost dimension is dense
template <typename T, int N>
bool encode_map(CUtensorMap* map, const void* base, const cuuint64_t (&sizes)[N],
                const int64_t (&strides)[N - 1], const cuuint32_t (&box)[N]) {
  const auto encode = encode_tiled();
  if (!encode) return false;
  cuuint64_t bytes[N - 1];
  cuuint32_t steps[N];
  for (int i = 0; i < N - 1; ++i) bytes[i] = (cuuint64_t)strides[i] * 2;
  for (int i = 0; i < N; ++i) steps[i] = 1;
  return encode(map,
                Half<T>::kExponent == 0x7F80u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                N, const_cast<void*>(base), sizes, bytes, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DV>
bool make_maps(LatentMaps* m, const LatentParams& p) {
  using L = Latent<DV>;
  const cuuint64_t width = p.width, page = p.page, blocks = p.n_blocks, B = p.B;
  const cuuint64_t rows = (cuuint64_t)p.nodes * p.heads;
  m->rows = wide_box_rows(p.page, 64);
  // keys in one copy a group, or in eight of eight rows where those are fewer than by chunks
  m->k_rows = m->rows == 64 ? 64 : m->rows <= 16 ? 8 : 0;
  const cuuint32_t run = m->rows, k_run = m->k_rows ? m->k_rows : 8;
  // a map takes the host half a microsecond: those that no copy uses are the values' once more
  auto whole = [&](CUtensorMap* map, cuuint32_t box_rows, cuuint32_t chunks) {
    return encode_map<T, 4>(map, p.k, {64, page, width / 64, blocks},
                            {p.token_stride, 64, p.block_stride}, {64, box_rows, chunks, 1});
  };
  bool ok = whole(&m->values, run, L::kVParts);
  m->tail = m->keys = m->q = m->values;
  if (m->k_rows) ok = ok && whole(&m->keys, k_run, L::kGroup);
  if (!m->k_rows || p.width % (64 * L::kGroup))
    ok = ok && encode_map<T, 3>(&m->tail, p.k, {width, page, blocks},
                                {p.token_stride, p.block_stride}, {64, run, 1});
  // Q by tensor copies where a request's rows are uniformly strided (and not broadcast); a negative
  // scale goes into its sign, which a copy cannot change
  const int64_t row = p.heads > 1 ? p.q_head : p.nodes > 1 ? p.q_node : p.width;
  const int64_t request = p.B > 1 ? p.q_req : row * (int64_t)rows;
  m->q_copies = p.scale2 >= 0.0f && (p.heads == 1 || p.nodes == 1 || p.q_node == row * p.heads) &&
                row > 0 && request > 0 && row < (1ll << 38) && request < (1ll << 38);
  if (m->q_copies)
    ok = ok && encode_map<T, 3>(&m->q, p.q, {width, rows, B}, {row, request}, {64, 64, 1});
  return ok;
}

template <typename T, int DV>
cudaError_t launch(const LatentParams& p, int sms, cudaStream_t stream) {
  using L = Latent<DV>;
  LatentMaps maps;
  if (!make_maps<T, DV>(&maps, p)) return cudaErrorInvalidValue;
  auto* kernel = latent_attention_kernel<T, DV>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const int pairs = min(kMaxPairs, max(1, sms / 2));
  kernel<<<2 * pairs, kLatentThreads, L::kSmem, stream>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while that one runs, waits on the device for its end
  cudaLaunchConfig_t cfg = {};
  constexpr int kRows = kLatentJoinThreads / 32 / (DV / 256);  // of a CTA
  cfg.gridDim = dim3(pairs, (p.part_rows + kRows - 1) / kRows);
  cfg.blockDim = dim3(kLatentJoinThreads);
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
  p.min_range = attn::kLatentMinRange;
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
