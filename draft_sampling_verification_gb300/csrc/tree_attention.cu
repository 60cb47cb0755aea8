// tree_attention.cu -- dspark_tree_attention: the nodes of a speculative step
// attend to their request's paged cache and to the nodes their tree shows.
// Host side; the kernels are in tree_attention.cuh.
#include "tree_attention.cuh"

namespace dspark {

int64_t tree_attention_workspace_bytes(int B, int nodes, int heads, int kv_heads, int head_dim) {
  // the more of what the two kernels want, as the blocks' size decides between them
  const int rows = nodes * (heads / kv_heads), cta_rows = attn::stream_rows(rows, head_dim);
  const int64_t streaming = attn::workspace_bytes(attn::part_rows(rows, cta_rows), head_dim,
                                                  attn::stream_ctas(head_dim, cta_rows));
  if (rows <= attn::few_rows(head_dim)) return streaming;
  const bool pair = head_dim != 256 && rows <= 128;
  const int64_t wide =
      attn::workspace_bytes(attn::part_rows(rows, head_dim == 256 || pair ? 128 : 256), head_dim,
                            attn::wide_ctas(pair));
  return streaming > wide ? streaming : wide;
}

cudaError_t launch_tree_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                  int64_t q_head, int B, int nodes, int heads, int kv_heads,
                                  int head_dim, const void* k, const void* v,
                                  int64_t block_stride, int64_t token_stride, int64_t head_stride,
                                  int n_blocks, int page, const int32_t* table, int64_t table_ld,
                                  int max_blocks, const int32_t* ctx, const int32_t* n_nodes,
                                  const uint64_t* mask, float scale, void* out, float* lse,
                                  int32_t* status, void* workspace, cudaStream_t stream) {
  attn::Params p;
  p.q = q;
  p.q_req = q_req;
  p.q_node = q_node;
  p.q_head = q_head;
  p.B = B;
  p.nodes = nodes;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
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
  p.scale2 = scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.workspace = static_cast<char*>(workspace);
  p.row_tiles = 1;
  p.min_range = attn::kMinRange;
  p.max_ctas = p.tile = p.item_cost = p.part_rows = p.part_wide = 0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (head_dim == 64) return attn::launch_64(p, dtype, sms, stream);
  if (head_dim == 128) return attn::launch_128(p, dtype, sms, stream);
  return attn::launch_256(p, dtype, sms, stream);
}

}  // namespace dspark
