// api.cu -- the extern "C" entry points declared in include/dspark.h.  Host
// code only: argument checks (nothing is launched on a bad argument), then
// one kernel launch on the caller's stream.  No allocation, no host sync.
#include <nvtx3/nvToolsExt.h>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "dspark.h"
#include "dspark_debug.h"

namespace dspark {
cudaError_t launch_q_topk(const void* x, int dtype, int64_t ld, int n_rows, int V,
                          const float* temperature, int top_k, uint32_t* counts, int32_t* ids,
                          int32_t* nnz, int32_t* status, int32_t* tokens, uint64_t seed,
                          const uint32_t* request_ids, int depth, cudaStream_t stream);
cudaError_t launch_q_dense(const void* x, int dtype, int64_t ld, int n_rows, int V,
                           const float* temperature, uint32_t* counts, int32_t* status,
                           int32_t* tokens, uint64_t seed, const uint32_t* request_ids, int depth,
                           cudaStream_t stream);
cudaError_t launch_draft_sample(const uint32_t* counts, const int32_t* ids, const int32_t* nnz,
                                int top_k, int B, int depth, int V, uint64_t seed,
                                const uint32_t* request_ids, int32_t* tokens, int32_t* status,
                                cudaStream_t stream);
cudaError_t launch_verify(int mode, const void* z, int dtype, int64_t ld, int B, int depth, int V,
                          const int32_t* drafts, const uint32_t* counts, const int32_t* ids,
                          const int32_t* nnz, int top_k, uint64_t seed,
                          const uint32_t* request_ids, int32_t* accept_len, int32_t* committed,
                          uint32_t* flags, int32_t* status, cudaStream_t stream);
cudaError_t launch_verify_modes(const void* z, int dtype, int64_t ld, int B, int depth, int V,
                                const int32_t* drafts, const uint32_t* counts, const int32_t* ids,
                                const int32_t* nnz, int top_k, uint64_t seed,
                                const uint32_t* request_ids, int32_t* g_acc, int32_t* g_com,
                                int32_t* g_st, int32_t* r_acc, int32_t* r_com, uint32_t* r_flags,
                                int32_t* r_st, cudaStream_t stream);
int spec_step_schedule(int B, int depth);
int64_t q_sharded_workspace_bytes(int n_rows);
cudaError_t launch_q_sharded(const void* x, int dtype, int64_t ld, int B, int depth, int V,
                             int n_sh, const float* temperature, int top_k, uint64_t seed,
                             const uint32_t* request_ids, uint32_t* counts, int32_t* ids,
                             int32_t* nnz, int32_t* tokens, int32_t* status, void* workspace,
                             cudaStream_t stream);
cudaError_t launch_q_chain(const void* x, int dtype, int64_t ld, int B, int depth, int V,
                           const float* temperature, const float* bias, int64_t bias_ld,
                           int n_bias, const int32_t* anchors, uint64_t seed,
                           const uint32_t* request_ids, uint32_t* counts, int32_t* tokens,
                           int32_t* status, float* margins, cudaStream_t stream);
cudaError_t launch_verify_match(const void* z, int dtype, int64_t ld, int B, int depth, int V,
                                const int32_t* drafts, uint64_t seed,
                                const uint32_t* request_ids, int32_t* accept_len,
                                int32_t* committed, uint32_t* flags, int32_t* status,
                                cudaStream_t stream);
cudaError_t launch_q_pack(const uint32_t* counts, const int32_t* ids, const int32_t* nnz,
                          int top_k, int n_rows, int V, float* q, uint64_t* checksum,
                          cudaStream_t stream);
cudaError_t launch_q_validate(const float* q, const int32_t* ids, const int32_t* nnz, int top_k,
                              int n_rows, int V, const int32_t* tokens, const uint64_t* expect,
                              uint32_t* counts, int32_t* status, cudaStream_t stream);
uint32_t* static_spec_workspace();
cudaError_t launch_spec_step(const void* xd, int d_dtype, int64_t ld_d, const void* xt,
                             int t_dtype, int64_t ld_t, int B, int depth, int V,
                             const float* temperature, uint64_t seed,
                             const uint32_t* request_ids, uint32_t* counts, int32_t* tokens,
                             int32_t* row_status, int32_t* g_acc, int32_t* g_com, int32_t* g_st,
                             int32_t* r_acc, int32_t* r_com, uint32_t* r_flags, int32_t* r_st,
                             uint32_t* workspace, int schedule, cudaStream_t stream);
cudaError_t launch_verify_stats(const uint32_t* flags, int B, uint32_t* stats,
                                cudaStream_t stream);
cudaError_t launch_target_probs(const void* z, int dtype, int64_t ld, int n_rows, int V,
                                float* p_out, int32_t* argmax, int32_t* status,
                                cudaStream_t stream);
cudaError_t launch_cache_plan(const int32_t* ctx, const int32_t* added, int B, int max_new,
                              int page, int32_t* table, int64_t table_ld, int max_blocks,
                              const int32_t* free_blocks, int max_free, const int32_t* n_free,
                              const int32_t* parents, int32_t* slots, int32_t* positions,
                              uint64_t* mask, int32_t* taken, int32_t* status,
                              cudaStream_t stream);
cudaError_t launch_kv_write(const void* k, const void* v, int src_dtype, int64_t src_token,
                            int64_t src_head, int n_src, int n_heads, int head_dim, void* k_cache,
                            void* v_cache, int cache_dtype, int64_t block_stride,
                            int64_t token_stride, int64_t head_stride, int n_blocks, int page,
                            const int32_t* slots, const int32_t* rows, int n_tokens,
                            cudaStream_t stream);
int64_t tree_attention_workspace_bytes(int B, int nodes, int heads, int kv_heads, int head_dim);
cudaError_t launch_tree_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                  int64_t q_head, int B, int nodes, int heads, int kv_heads,
                                  int head_dim, const void* k, const void* v,
                                  int64_t block_stride, int64_t token_stride, int64_t head_stride,
                                  int n_blocks, int page, const int32_t* table, int64_t table_ld,
                                  int max_blocks, const int32_t* ctx, const int32_t* n_nodes,
                                  const uint64_t* mask, float scale, void* out, float* lse,
                                  int32_t* status, void* workspace, cudaStream_t stream);
void rope_table(int rot_dim, double base, int scaling, double factor, double original_len,
                double low, double high, const double* inv_freq, uint64_t* table);
cudaError_t launch_rotate(const void* q, const void* k, const void* v, int src_dtype,
                          int64_t q_token, int64_t q_head, int64_t k_token, int64_t k_head,
                          int n_src, int n_tokens, int heads, int kv_heads, int dim,
                          const float* q_weight, const float* k_weight, float eps,
                          const int32_t* positions, const uint64_t* table, int rot_start,
                          int rot_dim, bool interleaved, float magnitude, void* q_out,
                          int64_t qo_token, int64_t qo_head, void* k_out, void* v_out,
                          int dst_dtype, int64_t block_stride, int64_t ko_token, int64_t ko_head,
                          int n_blocks, int page, const int32_t* slots, const int32_t* src_rows,
                          cudaStream_t stream);
cudaError_t launch_latent_write(const void* c, int64_t c_token, const void* r, int64_t r_token,
                                int src_dtype, int n_src, int latent, int rope,
                                const float* weight, float eps, const int32_t* positions,
                                const uint64_t* table, bool interleaved, float magnitude,
                                void* cache, int cache_dtype, int64_t block_stride,
                                int64_t token_stride, int n_blocks, int page,
                                const int32_t* slots, const int32_t* src_rows, int n_tokens,
                                cudaStream_t stream);
int64_t latent_attention_workspace_bytes(int B, int nodes, int heads, int latent);
cudaError_t launch_latent_attention(const void* q, int dtype, int64_t q_req, int64_t q_node,
                                    int64_t q_head, int B, int nodes, int heads, int latent,
                                    int rope, const void* cache, int64_t block_stride,
                                    int64_t token_stride, int n_blocks, int page,
                                    const int32_t* table, int64_t table_ld, int max_blocks,
                                    const int32_t* ctx, const int32_t* n_nodes,
                                    const uint64_t* mask, float scale, void* out, float* lse,
                                    int32_t* status, void* workspace, cudaStream_t stream);
cudaError_t launch_logits_process(
    const void* x, int dtype, int64_t ld, int B, int rows, int V, const int32_t* history,
    int64_t history_ld, const int32_t* prompt_len, const int32_t* history_len,
    const int32_t* drafts, int n_drafts, const uint64_t* row_mask, const float* repetition,
    const float* frequency, const float* presence, const int32_t* bias_ids,
    const float* bias_values, int max_bias, const int32_t* n_bias, const uint32_t* words,
    int64_t mask_ld, int n_masks, const int32_t* mask_rows, void* out, int64_t ld_out,
    int32_t* status, cudaStream_t stream);
#ifdef DSPARK_CHECKED
namespace attn {
cudaError_t stall_64(uint32_t v);
cudaError_t stall_128(uint32_t v);
cudaError_t stall_256(uint32_t v);
cudaError_t stall_latent(uint32_t v);
}  // namespace attn
cudaError_t dspark_check_collect_cache(uint32_t* out);
cudaError_t dspark_check_collect_tree_attention_64(uint32_t* out);
cudaError_t dspark_check_collect_tree_attention_128(uint32_t* out);
cudaError_t dspark_check_collect_tree_attention_256(uint32_t* out);
cudaError_t dspark_check_collect_logits(uint32_t* out);
cudaError_t dspark_check_collect_rotate(uint32_t* out);
cudaError_t dspark_check_collect_latent_attention(uint32_t* out);
cudaError_t dspark_check_collect_chain(uint32_t* out);
cudaError_t dspark_check_collect_debug(uint32_t* out);
cudaError_t dspark_check_collect_q_dense(uint32_t* out);
cudaError_t dspark_check_collect_q_topk(uint32_t* out);
cudaError_t dspark_check_collect_q_wire(uint32_t* out);
cudaError_t dspark_check_collect_sample(uint32_t* out);
cudaError_t dspark_check_collect_spec(uint32_t* out);
cudaError_t dspark_check_collect_tp(uint32_t* out);
cudaError_t dspark_check_collect_verify(uint32_t* out);
#endif
}  // namespace dspark

namespace {

// One NVTX range per ABI call, named after the call (a no-op unless a tool
// such as Nsight Systems is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr int kMaxGridRows = (1 << 30) / 8;  // rows per launch (8-CTA clusters)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int esize(int32_t dtype) { return dtype == DSPARK_F32 ? 4 : 2; }

int check_common(int32_t dtype, int32_t V, int64_t ld) {
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return DSPARK_ERR_DTYPE;
  if (V < 1 || V > DSPARK_MAX_V) return DSPARK_ERR_SIZE;
  if (ld < V) return DSPARK_ERR_SIZE;
  return 0;
}

int check_topk(int32_t top_k, int32_t V) {
  if (top_k < 0 || top_k > V || top_k > DSPARK_MAX_TOPK) return DSPARK_ERR_TOPK;
  return 0;
}

int launch_result(cudaError_t e) { return e == cudaSuccess ? 0 : (int)e; }

// `count` places, `stride` >= 0 elements apart
struct Dim {
  int64_t count, stride;
};

// Whether two different places of a layout share an element, `width` elements lying at each: whether
// steps along its dimensions that are not all 0 lead less than `width` from where they start.  From
// the last dimension to the first, only steps that the dimensions before it can make good: with
// dimensions in the order of their strides, none where each lies within one step of the next.
bool meets(const Dim* dims, int n, __int128 at, int64_t width, bool moved) {
  if (n == 0) return moved && at > -(__int128)width && at < width;
  const __int128 stride = dims[n - 1].stride, most = dims[n - 1].count - 1;
  __int128 reach = width - 1;
  for (int i = 0; i < n - 1; ++i) reach += (__int128)(dims[i].count - 1) * dims[i].stride;
  // at + k stride in [-reach, reach]
  const __int128 lo = -reach - at, hi = reach - at;
  __int128 first = lo / stride + (lo % stride > 0 ? 1 : 0);
  __int128 last = hi / stride - (hi % stride < 0 ? 1 : 0);
  first = first < -most ? -most : first;
  last = last > most ? most : last;
  for (__int128 k = first; k <= last; ++k)
    if (meets(dims, n - 1, at + k * stride, width, moved || k != 0)) return true;
  return false;
}
template <int N>
bool shares_places(const Dim (&all)[N], int64_t width) {
  Dim dims[N];
  int n = 0;
  for (const Dim& d : all)
    if (d.count < 1) return false;
  for (const Dim& d : all) {
    if (d.count == 1) continue;
    if (d.stride < width) return true;
    int i = n++;
    for (; i > 0 && dims[i - 1].stride > d.stride; --i) dims[i] = dims[i - 1];
    dims[i] = d;
  }
  return meets(dims, n, 0, width, false);
}

}  // namespace

extern "C" {

const char* dspark_version(void) { return "dspark-gb300 0.1 (" DSPARK_QSEM ", sm_103a)"; }

int dspark_checked_status(uint32_t* out) {
  if (!out) return DSPARK_ERR_NULL;
  out[0] = out[1] = 0u;
#ifdef DSPARK_CHECKED
  out[2] = 1u;
  cudaError_t e = cudaSuccess;
  cudaError_t (*collect[])(uint32_t*) = {
      dspark::dspark_check_collect_cache, dspark::dspark_check_collect_logits,
      dspark::dspark_check_collect_rotate, dspark::dspark_check_collect_latent_attention,
      dspark::dspark_check_collect_tree_attention_64,
      dspark::dspark_check_collect_tree_attention_128,
      dspark::dspark_check_collect_tree_attention_256,
      dspark::dspark_check_collect_chain, dspark::dspark_check_collect_debug,
      dspark::dspark_check_collect_q_dense, dspark::dspark_check_collect_q_topk,
      dspark::dspark_check_collect_q_wire, dspark::dspark_check_collect_sample,
      dspark::dspark_check_collect_spec, dspark::dspark_check_collect_tp,
      dspark::dspark_check_collect_verify};
  for (auto fn : collect)
    if (e == cudaSuccess) e = fn(out);
  return e == cudaSuccess ? 0 : (int)e;
#else
  out[2] = 0u;
  return 0;
#endif
}

int dspark_debug_stall_attention(int32_t cta) {
  if (cta < -1) return DSPARK_ERR_ARG;
#ifdef DSPARK_CHECKED
  const uint32_t v = (uint32_t)(cta + 1);
  for (auto set : {dspark::attn::stall_64, dspark::attn::stall_128, dspark::attn::stall_256,
                   dspark::attn::stall_latent})
    if (const cudaError_t e = set(v)) return (int)e;
  return 0;
#else
  return cta < 0 ? 0 : DSPARK_ERR_ARG;
#endif
}

int dspark_q_build(const void* draft_logits, int32_t dtype, int64_t ld, int32_t n_rows, int32_t V,
                   const float* temperature, int32_t top_k, uint32_t* counts, int32_t* sparse_ids,
                   int32_t* nnz, int32_t* row_status, void* stream) {
  const NvtxRange nvtx_range("dspark_q_build");
  if (int e = check_common(dtype, V, ld)) return e;
  if (int e = check_topk(top_k, V)) return e;
  if (n_rows < 0 || n_rows > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (n_rows == 0) return 0;
  if (!draft_logits || !counts || !row_status) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(draft_logits, esize(dtype)) || !aligned(counts, 4) || !aligned(row_status, 4) ||
      (temperature && !aligned(temperature, 4)) || (sparse_ids && !aligned(sparse_ids, 4)) ||
      (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  if (top_k == 0)
    return launch_result(dspark::launch_q_dense(draft_logits, dtype, ld, n_rows, V, temperature,
                                                counts, row_status, nullptr, 0ull, nullptr, 1,
                                                static_cast<cudaStream_t>(stream)));
  return launch_result(dspark::launch_q_topk(draft_logits, dtype, ld, n_rows, V, temperature,
                                             top_k, counts, sparse_ids, nnz, row_status, nullptr,
                                             0ull, nullptr, 1, static_cast<cudaStream_t>(stream)));
}

int dspark_q_build_sample(const void* draft_logits, int32_t dtype, int64_t ld, int32_t B,
                          int32_t depth, int32_t V, const float* temperature, int32_t top_k,
                          uint64_t seed, const uint32_t* request_ids, uint32_t* counts,
                          int32_t* sparse_ids, int32_t* nnz, int32_t* draft_tokens,
                          int32_t* row_status, void* stream) {
  const NvtxRange nvtx_range("dspark_q_build_sample");
  if (int e = check_common(dtype, V, ld)) return e;
  if (int e = check_topk(top_k, V)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (B == 0) return 0;
  if (!draft_logits || !counts || !row_status || !draft_tokens) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(draft_logits, esize(dtype)) || !aligned(counts, 4) || !aligned(row_status, 4) ||
      !aligned(draft_tokens, 4) || (temperature && !aligned(temperature, 4)) ||
      (sparse_ids && !aligned(sparse_ids, 4)) || (nnz && !aligned(nnz, 4)) ||
      (request_ids && !aligned(request_ids, 4)))
    return DSPARK_ERR_ALIGN;
  if (top_k == 0)
    return launch_result(dspark::launch_q_dense(draft_logits, dtype, ld, B * depth, V, temperature,
                                                counts, row_status, draft_tokens, seed,
                                                request_ids, depth,
                                                static_cast<cudaStream_t>(stream)));
  return launch_result(dspark::launch_q_topk(draft_logits, dtype, ld, B * depth, V, temperature,
                                             top_k, counts, sparse_ids, nnz, row_status,
                                             draft_tokens, seed, request_ids, depth,
                                             static_cast<cudaStream_t>(stream)));
}

int dspark_draft_sample(const uint32_t* counts, const int32_t* sparse_ids, const int32_t* nnz,
                        int32_t top_k, int32_t B, int32_t depth, int32_t V, uint64_t seed,
                        const uint32_t* request_ids, int32_t* draft_tokens, int32_t* row_status,
                        void* stream) {
  const NvtxRange nvtx_range("dspark_draft_sample");
  if (V < 1 || V > DSPARK_MAX_V) return DSPARK_ERR_SIZE;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth > (int64_t)(1 << 30)) return DSPARK_ERR_SIZE;
  if (int e = check_topk(top_k, V)) return e;
  if (B == 0) return 0;
  if (!counts || !draft_tokens || !row_status) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(counts, 4) || !aligned(draft_tokens, 4) || !aligned(row_status, 4) ||
      (request_ids && !aligned(request_ids, 4)) || (sparse_ids && !aligned(sparse_ids, 4)) ||
      (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_draft_sample(counts, sparse_ids, nnz, top_k, B, depth, V,
                                                   seed, request_ids, draft_tokens, row_status,
                                                   static_cast<cudaStream_t>(stream)));
}

static int check_verify(const void* target_logits, int32_t dtype, int64_t ld, int32_t B,
                        int32_t depth, int32_t V, const int32_t* draft_tokens,
                        const int32_t* accept_len, const int32_t* committed,
                        const int32_t* req_status) {
  if (int e = check_common(dtype, V, ld)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || B > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (B == 0) return 1;  // nothing to do
  if (!target_logits || !draft_tokens || !accept_len || !committed || !req_status)
    return DSPARK_ERR_NULL;
  if (!aligned(target_logits, esize(dtype)) || !aligned(draft_tokens, 4) ||
      !aligned(accept_len, 4) || !aligned(committed, 4) || !aligned(req_status, 4))
    return DSPARK_ERR_ALIGN;
  return 0;
}

int dspark_verify_greedy(const void* target_logits, int32_t dtype, int64_t ld, int32_t B,
                         int32_t depth, int32_t V, const int32_t* draft_tokens,
                         int32_t* accept_len, int32_t* committed, int32_t* req_status,
                         void* stream) {
  const NvtxRange nvtx_range("dspark_verify_greedy");
  const int e = check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens, accept_len,
                             committed, req_status);
  if (e != 0) return e > 0 ? 0 : e;
  return launch_result(dspark::launch_verify(0, target_logits, dtype, ld, B, depth, V,
                                             draft_tokens, nullptr, nullptr, nullptr, 0, 0ull,
                                             nullptr, accept_len, committed, nullptr, req_status,
                                             static_cast<cudaStream_t>(stream)));
}

int dspark_verify_ratio(const void* target_logits, int32_t dtype, int64_t ld, int32_t B,
                        int32_t depth, int32_t V, const int32_t* draft_tokens,
                        const uint32_t* counts, const int32_t* sparse_ids, const int32_t* nnz,
                        int32_t top_k, uint64_t seed, const uint32_t* request_ids,
                        int32_t* accept_len, int32_t* committed, uint32_t* flags,
                        int32_t* req_status, void* stream) {
  const NvtxRange nvtx_range("dspark_verify_ratio");
  const int e = check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens, accept_len,
                             committed, req_status);
  if (e != 0) return e > 0 ? 0 : e;
  if (int e2 = check_topk(top_k, V)) return e2;
  if (!counts) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(counts, 4) || (flags && !aligned(flags, 4)) ||
      (request_ids && !aligned(request_ids, 4)) || (sparse_ids && !aligned(sparse_ids, 4)) ||
      (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_verify(1, target_logits, dtype, ld, B, depth, V,
                                             draft_tokens, counts, sparse_ids, nnz, top_k, seed,
                                             request_ids, accept_len, committed, flags,
                                             req_status, static_cast<cudaStream_t>(stream)));
}

int dspark_verify_match(const void* target_logits, int32_t dtype, int64_t ld, int32_t B,
                        int32_t depth, int32_t V, const int32_t* draft_tokens, uint64_t seed,
                        const uint32_t* request_ids, int32_t* accept_len, int32_t* committed,
                        uint32_t* flags, int32_t* req_status, void* stream) {
  const NvtxRange nvtx_range("dspark_verify_match");
  const int e = check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens, accept_len,
                             committed, req_status);
  if (e != 0) return e > 0 ? 0 : e;
  if ((flags && !aligned(flags, 4)) || (request_ids && !aligned(request_ids, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_verify_match(target_logits, dtype, ld, B, depth, V,
                                                   draft_tokens, seed, request_ids, accept_len,
                                                   committed, flags, req_status,
                                                   static_cast<cudaStream_t>(stream)));
}

int dspark_verify(const void* target_logits, int32_t dtype, int64_t ld, int32_t B, int32_t depth,
                  int32_t V, const int32_t* draft_tokens, const uint32_t* counts,
                  const int32_t* sparse_ids, const int32_t* nnz, int32_t top_k, uint64_t seed,
                  const uint32_t* request_ids, int32_t* greedy_accept_len,
                  int32_t* greedy_committed, int32_t* greedy_status, int32_t* ratio_accept_len,
                  int32_t* ratio_committed, uint32_t* ratio_flags, int32_t* ratio_status,
                  void* stream) {
  const NvtxRange nvtx_range("dspark_verify");
  const bool g = greedy_accept_len || greedy_committed || greedy_status;
  const bool r = ratio_accept_len || ratio_committed || ratio_status;
  if (!g && !r) return DSPARK_ERR_NULL;
  if (g && (!greedy_accept_len || !greedy_committed || !greedy_status)) return DSPARK_ERR_NULL;
  int e = g ? check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens,
                           greedy_accept_len, greedy_committed, greedy_status)
            : check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens, ratio_accept_len,
                           ratio_committed, ratio_status);
  if (e != 0) return e > 0 ? 0 : e;  // > 0: empty batch
  if (r) {
    const int e2 = check_verify(target_logits, dtype, ld, B, depth, V, draft_tokens,
                                ratio_accept_len, ratio_committed, ratio_status);
    if (e2 < 0) return e2;
    if (int e3 = check_topk(top_k, V)) return e3;
    if (!counts) return DSPARK_ERR_NULL;
    if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
    if (!aligned(counts, 4) || (ratio_flags && !aligned(ratio_flags, 4)) ||
        (request_ids && !aligned(request_ids, 4)) || (sparse_ids && !aligned(sparse_ids, 4)) ||
        (nnz && !aligned(nnz, 4)))
      return DSPARK_ERR_ALIGN;
  }
  return launch_result(dspark::launch_verify_modes(
      target_logits, dtype, ld, B, depth, V, draft_tokens, r ? counts : nullptr,
      r ? sparse_ids : nullptr, r ? nnz : nullptr, r ? top_k : 0, seed, request_ids,
      g ? greedy_accept_len : nullptr, greedy_committed, greedy_status,
      r ? ratio_accept_len : nullptr, ratio_committed, ratio_flags, ratio_status,
      static_cast<cudaStream_t>(stream)));
}

int dspark_spec_step_schedule(int32_t B, int32_t depth) {
  if (B < 0 || depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  return dspark::spec_step_schedule(B, depth);
}

static int spec_step_impl(const void* draft_logits, int32_t draft_dtype, int64_t ld_draft,
                          const void* target_logits, int32_t target_dtype, int64_t ld_target,
                          int32_t B, int32_t depth, int32_t V, const float* temperature,
                          uint64_t seed, const uint32_t* request_ids, uint32_t* counts,
                          int32_t* draft_tokens, int32_t* row_status, int32_t* greedy_accept_len,
                          int32_t* greedy_committed, int32_t* greedy_status,
                          int32_t* ratio_accept_len, int32_t* ratio_committed,
                          uint32_t* ratio_flags, int32_t* ratio_status, uint32_t* workspace,
                          bool static_workspace, int32_t schedule, void* stream) {
  if (int e = check_common(draft_dtype, V, ld_draft)) return e;
  if (int e = check_common(target_dtype, V, ld_target)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (schedule < DSPARK_SCHEDULE_AUTO || schedule > DSPARK_SCHEDULE_SEPARATE)
    return DSPARK_ERR_ARG;
  if (B == 0) return 0;
  const bool g = greedy_accept_len || greedy_committed || greedy_status;
  const bool r = ratio_accept_len || ratio_committed || ratio_status;
  if (!draft_logits || !target_logits || !counts || !draft_tokens || !row_status)
    return DSPARK_ERR_NULL;
  if (!workspace && !static_workspace) return DSPARK_ERR_NULL;
  if (!g && !r) return DSPARK_ERR_NULL;
  if (g && (!greedy_accept_len || !greedy_committed || !greedy_status)) return DSPARK_ERR_NULL;
  if (r && (!ratio_accept_len || !ratio_committed || !ratio_status)) return DSPARK_ERR_NULL;
  const void* four[] = {counts, draft_tokens, row_status, greedy_accept_len, greedy_committed,
                        greedy_status, ratio_accept_len, ratio_committed, ratio_flags,
                        ratio_status, temperature, request_ids, workspace};
  for (const void* q : four)
    if (q && !aligned(q, 4)) return DSPARK_ERR_ALIGN;
  if (!aligned(draft_logits, esize(draft_dtype)) || !aligned(target_logits, esize(target_dtype)))
    return DSPARK_ERR_ALIGN;
  if (static_workspace) {
    if (B > DSPARK_SPEC_STATIC_MAX_B) return DSPARK_ERR_SIZE;
    if ((workspace = dspark::static_spec_workspace()) == nullptr) return DSPARK_ERR_DEVICE;
  }
  return launch_result(dspark::launch_spec_step(
      draft_logits, draft_dtype, ld_draft, target_logits, target_dtype, ld_target, B, depth, V,
      temperature, seed, request_ids, counts, draft_tokens, row_status,
      g ? greedy_accept_len : nullptr, greedy_committed, greedy_status,
      r ? ratio_accept_len : nullptr, ratio_committed, ratio_flags, ratio_status, workspace,
      schedule, static_cast<cudaStream_t>(stream)));
}

int dspark_spec_step(const void* draft_logits, int32_t draft_dtype, int64_t ld_draft,
                     const void* target_logits, int32_t target_dtype, int64_t ld_target,
                     int32_t B, int32_t depth, int32_t V, const float* temperature, uint64_t seed,
                     const uint32_t* request_ids, uint32_t* counts, int32_t* draft_tokens,
                     int32_t* row_status, int32_t* greedy_accept_len, int32_t* greedy_committed,
                     int32_t* greedy_status, int32_t* ratio_accept_len, int32_t* ratio_committed,
                     uint32_t* ratio_flags, int32_t* ratio_status, uint32_t* workspace,
                     int32_t schedule, void* stream) {
  const NvtxRange nvtx_range("dspark_spec_step");
  return spec_step_impl(draft_logits, draft_dtype, ld_draft, target_logits, target_dtype,
                        ld_target, B, depth, V, temperature, seed, request_ids, counts,
                        draft_tokens, row_status, greedy_accept_len, greedy_committed,
                        greedy_status, ratio_accept_len, ratio_committed, ratio_flags,
                        ratio_status, workspace, false, schedule, stream);
}

int dspark_spec_step_noalloc(const void* draft_logits, int32_t draft_dtype, int64_t ld_draft,
                             const void* target_logits, int32_t target_dtype, int64_t ld_target,
                             int32_t B, int32_t depth, int32_t V, const float* temperature,
                             uint64_t seed, const uint32_t* request_ids, uint32_t* counts,
                             int32_t* draft_tokens, int32_t* row_status,
                             int32_t* greedy_accept_len, int32_t* greedy_committed,
                             int32_t* greedy_status, int32_t* ratio_accept_len,
                             int32_t* ratio_committed, uint32_t* ratio_flags,
                             int32_t* ratio_status, int32_t schedule, void* stream) {
  const NvtxRange nvtx_range("dspark_spec_step_noalloc");
  return spec_step_impl(draft_logits, draft_dtype, ld_draft, target_logits, target_dtype,
                        ld_target, B, depth, V, temperature, seed, request_ids, counts,
                        draft_tokens, row_status, greedy_accept_len, greedy_committed,
                        greedy_status, ratio_accept_len, ratio_committed, ratio_flags,
                        ratio_status, nullptr, true, schedule, stream);
}

namespace {

// The staging buffer of dspark_spec_step_host: 256-byte aligned segments.
struct HostStaging {
  int64_t counts, draft, target, temperature, request_ids, tokens, row_status, g_acc, g_com,
      g_st, r_acc, r_com, r_flags, r_st, workspace, total;
};

int64_t seg(int64_t* at, int64_t bytes) {
  const int64_t o = *at;
  *at += (bytes + 255) / 256 * 256;
  return o;
}

HostStaging host_staging(int32_t B, int32_t depth, int32_t V, int32_t dd, int32_t td) {
  HostStaging h;
  int64_t at = 0;
  const int64_t rows = (int64_t)B * depth, trows = (int64_t)B * (depth + 1);
  h.counts = seg(&at, rows * V * 4);
  h.draft = seg(&at, rows * V * esize(dd));
  h.target = seg(&at, trows * V * esize(td));
  h.temperature = seg(&at, rows * 4);
  h.request_ids = seg(&at, (int64_t)B * 4);
  h.tokens = seg(&at, rows * 4);
  h.row_status = seg(&at, rows * 4);
  h.g_acc = seg(&at, (int64_t)B * 4);
  h.g_com = seg(&at, trows * 4);
  h.g_st = seg(&at, (int64_t)B * 4);
  h.r_acc = seg(&at, (int64_t)B * 4);
  h.r_com = seg(&at, trows * 4);
  h.r_flags = seg(&at, (int64_t)B * 4);
  h.r_st = seg(&at, (int64_t)B * 4);
  h.workspace = seg(&at, ((int64_t)B + 1) * 4);
  h.total = at;
  return h;
}

}  // namespace

int64_t dspark_spec_step_host_staging_bytes(int32_t B, int32_t depth, int32_t V,
                                            int32_t draft_dtype, int32_t target_dtype) {
  if (B < 0 || depth < 1 || depth > DSPARK_MAX_DEPTH || V < 1 || V > DSPARK_MAX_V) return 0;
  if (check_common(draft_dtype, V, V) || check_common(target_dtype, V, V)) return 0;
  return host_staging(B, depth, V, draft_dtype, target_dtype).total;
}

int dspark_spec_step_host(const void* h_draft_logits, int32_t draft_dtype,
                          const void* h_target_logits, int32_t target_dtype, int32_t B,
                          int32_t depth, int32_t V, const float* h_temperature, uint64_t seed,
                          const uint32_t* h_request_ids, int32_t* h_draft_tokens,
                          int32_t* h_row_status, int32_t* h_greedy_accept_len,
                          int32_t* h_greedy_committed, int32_t* h_greedy_status,
                          int32_t* h_ratio_accept_len, int32_t* h_ratio_committed,
                          uint32_t* h_ratio_flags, int32_t* h_ratio_status, void* staging,
                          int32_t schedule, void* stream) {
  const NvtxRange nvtx_range("dspark_spec_step_host");
  if (int e = check_common(draft_dtype, V, V)) return e;
  if (int e = check_common(target_dtype, V, V)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (schedule < DSPARK_SCHEDULE_AUTO || schedule > DSPARK_SCHEDULE_SEPARATE)
    return DSPARK_ERR_ARG;
  if (B == 0) return 0;
  const bool g = h_greedy_accept_len || h_greedy_committed || h_greedy_status;
  const bool r = h_ratio_accept_len || h_ratio_committed || h_ratio_status;
  if (!h_draft_logits || !h_target_logits || !h_draft_tokens || !h_row_status || !staging)
    return DSPARK_ERR_NULL;
  if (!g && !r) return DSPARK_ERR_NULL;
  if (g && (!h_greedy_accept_len || !h_greedy_committed || !h_greedy_status))
    return DSPARK_ERR_NULL;
  if (r && (!h_ratio_accept_len || !h_ratio_committed || !h_ratio_status)) return DSPARK_ERR_NULL;
  if (!aligned(staging, 256)) return DSPARK_ERR_ALIGN;
  const HostStaging h = host_staging(B, depth, V, draft_dtype, target_dtype);
  char* base = static_cast<char*>(staging);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)B * depth, trows = (int64_t)B * (depth + 1);
  auto h2d = [&](int64_t off, const void* src, int64_t bytes) {
    return cudaMemcpyAsync(base + off, src, (size_t)bytes, cudaMemcpyHostToDevice, st);
  };
  auto d2h = [&](void* dst, int64_t off, int64_t bytes) {
    return cudaMemcpyAsync(dst, base + off, (size_t)bytes, cudaMemcpyDeviceToHost, st);
  };
  cudaError_t e = h2d(h.draft, h_draft_logits, rows * V * esize(draft_dtype));
  if (e == cudaSuccess) e = h2d(h.target, h_target_logits, trows * V * esize(target_dtype));
  if (e == cudaSuccess && h_temperature) e = h2d(h.temperature, h_temperature, rows * 4);
  if (e == cudaSuccess && h_request_ids) e = h2d(h.request_ids, h_request_ids, (int64_t)B * 4);
  if (e != cudaSuccess) return launch_result(e);
  auto dp = [&](int64_t off) { return reinterpret_cast<int32_t*>(base + off); };
  const int rc = spec_step_impl(
      base + h.draft, draft_dtype, V, base + h.target, target_dtype, V, B, depth, V,
      h_temperature ? reinterpret_cast<const float*>(base + h.temperature) : nullptr, seed,
      h_request_ids ? reinterpret_cast<const uint32_t*>(base + h.request_ids) : nullptr,
      reinterpret_cast<uint32_t*>(base + h.counts), dp(h.tokens), dp(h.row_status),
      g ? dp(h.g_acc) : nullptr, g ? dp(h.g_com) : nullptr, g ? dp(h.g_st) : nullptr,
      r ? dp(h.r_acc) : nullptr, r ? dp(h.r_com) : nullptr,
      (r && h_ratio_flags) ? reinterpret_cast<uint32_t*>(base + h.r_flags) : nullptr,
      r ? dp(h.r_st) : nullptr, reinterpret_cast<uint32_t*>(base + h.workspace), false, schedule,
      stream);
  if (rc != 0) return rc;
  e = d2h(h_draft_tokens, h.tokens, rows * 4);
  if (e == cudaSuccess) e = d2h(h_row_status, h.row_status, rows * 4);
  if (e == cudaSuccess && g) e = d2h(h_greedy_accept_len, h.g_acc, (int64_t)B * 4);
  if (e == cudaSuccess && g) e = d2h(h_greedy_committed, h.g_com, trows * 4);
  if (e == cudaSuccess && g) e = d2h(h_greedy_status, h.g_st, (int64_t)B * 4);
  if (e == cudaSuccess && r) e = d2h(h_ratio_accept_len, h.r_acc, (int64_t)B * 4);
  if (e == cudaSuccess && r) e = d2h(h_ratio_committed, h.r_com, trows * 4);
  if (e == cudaSuccess && r && h_ratio_flags) e = d2h(h_ratio_flags, h.r_flags, (int64_t)B * 4);
  if (e == cudaSuccess && r) e = d2h(h_ratio_status, h.r_st, (int64_t)B * 4);
  return launch_result(e);
}

int dspark_q_chain_sample(const void* draft_logits, int32_t dtype, int64_t ld, int32_t B,
                          int32_t depth, int32_t V, const float* temperature, const float* bias,
                          int64_t bias_ld, int32_t n_bias, const int32_t* anchors, uint64_t seed,
                          const uint32_t* request_ids, float* workspace, uint32_t* counts,
                          int32_t* draft_tokens, int32_t* row_status, float* margins,
                          void* stream) {
  const NvtxRange nvtx_range("dspark_q_chain_sample");
  if (int e = check_common(dtype, V, ld)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (bias && (n_bias < 1 || bias_ld < V)) return DSPARK_ERR_SIZE;
  if (B == 0) return 0;
  // the workspace is no longer used (z is formed in shared memory); it may be NULL
  if (!draft_logits || !anchors || !counts || !draft_tokens || !row_status)
    return DSPARK_ERR_NULL;
  const void* four[] = {anchors, workspace, counts, draft_tokens, row_status, margins,
                        temperature, request_ids, bias};
  for (const void* q : four)
    if (q && !aligned(q, 4)) return DSPARK_ERR_ALIGN;
  if (!aligned(draft_logits, esize(dtype))) return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_q_chain(
      draft_logits, dtype, ld, B, depth, V, temperature, bias, bias_ld, bias ? n_bias : 1,
      anchors, seed, request_ids, counts, draft_tokens, row_status, margins,
      static_cast<cudaStream_t>(stream)));
}

int64_t dspark_q_sharded_workspace_bytes(int32_t n_rows) {
  return n_rows < 0 ? 0 : dspark::q_sharded_workspace_bytes(n_rows);
}

int dspark_q_build_sample_sharded(const void* draft_logits, int32_t dtype, int64_t ld, int32_t B,
                                  int32_t depth, int32_t V, int32_t n_shards,
                                  const float* temperature, int32_t top_k, uint64_t seed,
                                  const uint32_t* request_ids, uint32_t* counts,
                                  int32_t* sparse_ids, int32_t* nnz, int32_t* draft_tokens,
                                  int32_t* row_status, void* workspace, void* stream) {
  const NvtxRange nvtx_range("dspark_q_build_sample_sharded");
  if (int e = check_common(dtype, V, ld)) return e;
  if (int e = check_topk(top_k, V)) return e;
  if (depth < 1 || depth > DSPARK_MAX_DEPTH) return DSPARK_ERR_SIZE;
  if (B < 0 || (int64_t)B * depth * 8 > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (n_shards < 1 || n_shards > 8) return DSPARK_ERR_ARG;
  if (B == 0) return 0;
  if (!draft_logits || !counts || !row_status || !workspace) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(draft_logits, esize(dtype)) || !aligned(counts, 4) || !aligned(row_status, 4) ||
      !aligned(workspace, 16) || (draft_tokens && !aligned(draft_tokens, 4)) ||
      (temperature && !aligned(temperature, 4)) || (request_ids && !aligned(request_ids, 4)) ||
      (sparse_ids && !aligned(sparse_ids, 4)) || (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_q_sharded(
      draft_logits, dtype, ld, B, depth, V, n_shards, temperature, top_k, seed, request_ids,
      counts, sparse_ids, nnz, draft_tokens, row_status, workspace,
      static_cast<cudaStream_t>(stream)));
}

int dspark_q_pack(const uint32_t* counts, const int32_t* sparse_ids, const int32_t* nnz,
                  int32_t top_k, int32_t n_rows, int32_t V, float* q_out,
                  uint64_t* checksum_out, void* stream) {
  const NvtxRange nvtx_range("dspark_q_pack");
  if (V < 1 || V > DSPARK_MAX_V) return DSPARK_ERR_SIZE;
  if (int e = check_topk(top_k, V)) return e;
  if (n_rows < 0 || n_rows > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (n_rows == 0) return 0;
  if (!counts || !q_out || !checksum_out) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(counts, 4) || !aligned(q_out, 4) || !aligned(checksum_out, 8) ||
      (sparse_ids && !aligned(sparse_ids, 4)) || (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_q_pack(counts, top_k > 0 ? sparse_ids : nullptr,
                                             top_k > 0 ? nnz : nullptr, top_k, n_rows, V, q_out,
                                             checksum_out, static_cast<cudaStream_t>(stream)));
}

int dspark_q_validate(const float* q, const int32_t* sparse_ids, const int32_t* nnz,
                      int32_t top_k, int32_t n_rows, int32_t V, const int32_t* tokens,
                      const uint64_t* expect, uint32_t* counts_out, int32_t* row_status,
                      void* stream) {
  const NvtxRange nvtx_range("dspark_q_validate");
  if (V < 1 || V > DSPARK_MAX_V) return DSPARK_ERR_SIZE;
  if (int e = check_topk(top_k, V)) return e;
  if (n_rows < 0 || n_rows > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (n_rows == 0) return 0;
  if (!q || !row_status) return DSPARK_ERR_NULL;
  if (top_k > 0 && (!sparse_ids || !nnz)) return DSPARK_ERR_NULL;
  if (!aligned(q, 4) || !aligned(row_status, 4) || (counts_out && !aligned(counts_out, 4)) ||
      (tokens && !aligned(tokens, 4)) || (expect && !aligned(expect, 8)) ||
      (sparse_ids && !aligned(sparse_ids, 4)) || (nnz && !aligned(nnz, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_q_validate(
      q, top_k > 0 ? sparse_ids : nullptr, top_k > 0 ? nnz : nullptr, top_k, n_rows, V, tokens,
      expect, counts_out, row_status, static_cast<cudaStream_t>(stream)));
}

int dspark_verify_stats(const uint32_t* flags, int32_t B, uint32_t* stats, void* stream) {
  const NvtxRange nvtx_range("dspark_verify_stats");
  if (B < 0 || B > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (!stats || (B > 0 && !flags)) return DSPARK_ERR_NULL;
  if (!aligned(stats, 4) || (flags && !aligned(flags, 4))) return DSPARK_ERR_ALIGN;
  return launch_result(
      dspark::launch_verify_stats(flags, B, stats, static_cast<cudaStream_t>(stream)));
}

int dspark_target_probs(const void* target_logits, int32_t dtype, int64_t ld, int32_t n_rows,
                        int32_t V, float* p_out, int32_t* argmax, int32_t* row_status,
                        void* stream) {
  const NvtxRange nvtx_range("dspark_target_probs");
  if (int e = check_common(dtype, V, ld)) return e;
  if (n_rows < 0 || n_rows > kMaxGridRows) return DSPARK_ERR_SIZE;
  if (n_rows == 0) return 0;
  if (!target_logits || !row_status) return DSPARK_ERR_NULL;
  if (!aligned(target_logits, esize(dtype)) || !aligned(row_status, 4) ||
      (p_out && !aligned(p_out, 4)) || (argmax && !aligned(argmax, 4)))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_target_probs(target_logits, dtype, ld, n_rows, V, p_out,
                                                   argmax, row_status,
                                                   static_cast<cudaStream_t>(stream)));
}

static bool aligned_or_null(const void* p, uintptr_t a) { return !p || aligned(p, a); }

// every address of a paged cache fits 63 bits and its slots 31
static int check_cache(int32_t n_blocks, int32_t page_size, int32_t cache_dtype,
                       int64_t block_stride, int64_t token_stride, int64_t head_stride) {
  if (cache_dtype != DSPARK_BF16 && cache_dtype != DSPARK_F16) return DSPARK_ERR_DTYPE;
  if (n_blocks < 1 || page_size < 1 || page_size > DSPARK_MAX_PAGE ||
      (int64_t)n_blocks * page_size > INT32_MAX)
    return DSPARK_ERR_SIZE;
  if (block_stride < 0 || token_stride < 0 || head_stride < 0) return DSPARK_ERR_SIZE;
  if (block_stride % 8 || token_stride % 8 || head_stride % 8) return DSPARK_ERR_ALIGN;
  return 0;
}

int dspark_cache_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t B, int32_t max_new,
                      int32_t page_size, int32_t* block_table, int64_t table_ld,
                      int32_t max_blocks, const int32_t* free_blocks, int32_t max_free,
                      const int32_t* n_free, const int32_t* parents, int32_t* slots,
                      int32_t* positions, uint64_t* tree_mask, int32_t* taken,
                      int32_t* req_status, void* stream) {
  const NvtxRange nvtx_range("dspark_cache_plan");
  if (B < 0 || B > DSPARK_MAX_PLANNED || max_new < 1 || page_size < 1 ||
      page_size > DSPARK_MAX_PAGE || max_blocks < 1 ||
      table_ld < max_blocks || max_free < 0 ||
      (int64_t)max_blocks * page_size > DSPARK_MAX_TOKENS ||
      max_new > (1 << 24) || (int64_t)B * max_new > INT32_MAX)
    return DSPARK_ERR_SIZE;
  if ((parents || tree_mask) && max_new > DSPARK_MAX_NODES) return DSPARK_ERR_SIZE;
  if (B == 0) return 0;
  if (!ctx_len || !new_len || !block_table || (max_free > 0 && !free_blocks) || !slots || !taken ||
      !req_status)
    return DSPARK_ERR_NULL;
  if (!aligned(ctx_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) ||
      !aligned_or_null(free_blocks, 4) || !aligned_or_null(n_free, 4) ||
      !aligned_or_null(parents, 4) || !aligned(slots, 4) || !aligned_or_null(positions, 4) ||
      !aligned_or_null(tree_mask, 8) || !aligned(taken, 4) || !aligned(req_status, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_cache_plan(
      ctx_len, new_len, B, max_new, page_size, block_table, table_ld, max_blocks, free_blocks,
      max_free, n_free, parents, slots, positions, tree_mask, taken, req_status,
      static_cast<cudaStream_t>(stream)));
}

int dspark_kv_write(const void* k, const void* v, int32_t src_dtype, int64_t src_token_stride,
                    int64_t src_head_stride, int32_t n_src, int32_t n_heads, int32_t head_dim,
                    void* k_cache, void* v_cache, int32_t cache_dtype, int64_t block_stride,
                    int64_t token_stride, int64_t head_stride, int32_t n_blocks,
                    int32_t page_size, const int32_t* slots, const int32_t* rows,
                    int32_t n_tokens, void* stream) {
  const NvtxRange nvtx_range("dspark_kv_write");
  if (int e = check_cache(n_blocks, page_size, cache_dtype, block_stride, token_stride,
                          head_stride))
    return e;
  if (src_dtype != DSPARK_F32 && src_dtype != cache_dtype) return DSPARK_ERR_DTYPE;
  if (n_src < 0 || n_tokens < 0 || n_heads < 1 || n_heads > 65535 || head_dim < 8 ||
      head_dim > 1024 || head_dim % 8 || src_token_stride < 0 || src_head_stride < 0)
    return DSPARK_ERR_SIZE;
  if (n_tokens == 0 || n_src == 0) return 0;
  if (!k || !v || !k_cache || !v_cache || !slots) return DSPARK_ERR_NULL;
  const int unit = src_dtype == DSPARK_F32 ? 4 : 8;
  if (src_token_stride % unit || src_head_stride % unit || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 4) ||
      !aligned_or_null(rows, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_kv_write(
      k, v, src_dtype, src_token_stride, src_head_stride, n_src, n_heads, head_dim, k_cache,
      v_cache, cache_dtype, block_stride, token_stride, head_stride, n_blocks, page_size, slots,
      rows, n_tokens, static_cast<cudaStream_t>(stream)));
}

static int check_heads(int32_t B, int32_t nodes, int32_t n_heads, int32_t n_kv_heads,
                       int32_t head_dim) {
  if (B < 0 || B > 65535 || nodes < 1 || nodes > DSPARK_MAX_NODES || n_kv_heads < 1 ||
      n_kv_heads > 1024 || n_heads < n_kv_heads || n_heads % n_kv_heads ||
      n_heads / n_kv_heads > 64 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return DSPARK_ERR_SIZE;
  return 0;
}

int64_t dspark_tree_attention_workspace_bytes(int32_t B, int32_t nodes, int32_t n_heads,
                                              int32_t n_kv_heads, int32_t head_dim) {
  if (check_heads(B, nodes, n_heads, n_kv_heads, head_dim)) return 0;
  return dspark::tree_attention_workspace_bytes(B, nodes, n_heads, n_kv_heads, head_dim);
}

int dspark_tree_attention(const void* q, int32_t dtype, int64_t q_req_stride,
                          int64_t q_node_stride, int64_t q_head_stride, int32_t B, int32_t nodes,
                          int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                          const void* k_cache, const void* v_cache, int64_t block_stride,
                          int64_t token_stride, int64_t head_stride, int32_t n_blocks,
                          int32_t page_size, const int32_t* block_table, int64_t table_ld,
                          int32_t max_blocks, const int32_t* ctx_len, const int32_t* n_nodes,
                          const uint64_t* tree_mask, float scale, void* out, float* lse,
                          int32_t* req_status, void* workspace, void* stream) {
  const NvtxRange nvtx_range("dspark_tree_attention");
  if (int e = check_cache(n_blocks, page_size, dtype, block_stride, token_stride, head_stride))
    return e;
  if (int e = check_heads(B, nodes, n_heads, n_kv_heads, head_dim)) return e;
  if (max_blocks < 1 || table_ld < max_blocks ||
      (int64_t)max_blocks * page_size > DSPARK_MAX_TOKENS ||
      q_req_stride < 0 || q_node_stride < 0 || q_head_stride < 0)
    return DSPARK_ERR_SIZE;
  // times log2(e) it has to stay finite, or a score of 0 would become NaN
  if (!(scale > -2.3e38f && scale < 2.3e38f)) return DSPARK_ERR_ARG;
  if (B == 0) return 0;
  if (!q || !k_cache || !v_cache || !block_table || !ctx_len || !n_nodes || !out || !req_status ||
      !workspace)
    return DSPARK_ERR_NULL;
  if (q_req_stride % 8 || q_node_stride % 8 || q_head_stride % 8 || !aligned(q, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(block_table, 4) || !aligned(ctx_len, 4) ||
      !aligned(n_nodes, 4) || !aligned_or_null(tree_mask, 8) || !aligned_or_null(lse, 4) ||
      !aligned(req_status, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_tree_attention(
      q, dtype, q_req_stride, q_node_stride, q_head_stride, B, nodes, n_heads, n_kv_heads,
      head_dim, k_cache, v_cache, block_stride, token_stride, head_stride, n_blocks, page_size,
      block_table, table_ld, max_blocks, ctx_len, n_nodes, tree_mask, scale, out, lse, req_status,
      workspace, static_cast<cudaStream_t>(stream)));
}

static bool positive(double v) { return v > 0.0 && v <= DBL_MAX; }

int dspark_rope_table(int32_t rot_dim, double base, int32_t scaling, double factor,
                      double original_len, double low, double high, const double* inv_freq,
                      uint64_t* table) {
  if (rot_dim < 8 || rot_dim > DSPARK_MAX_HEAD || rot_dim % 8) return DSPARK_ERR_SIZE;
  if (!table) return DSPARK_ERR_NULL;
  if (!aligned(table, 8) || !aligned_or_null(inv_freq, 8)) return DSPARK_ERR_ALIGN;
  if (scaling < DSPARK_ROPE_PLAIN || scaling > DSPARK_ROPE_PARTS) return DSPARK_ERR_ARG;
  if (!inv_freq && !positive(base)) return DSPARK_ERR_ARG;
  if (scaling != DSPARK_ROPE_PLAIN && !positive(factor)) return DSPARK_ERR_ARG;
  if (scaling == DSPARK_ROPE_PARTS &&
      (!positive(original_len) || !positive(high - low) || !(low >= -DBL_MAX && low <= DBL_MAX)))
    return DSPARK_ERR_ARG;
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    const double f = inv_freq ? inv_freq[i] : std::pow(base, -2.0 * i / rot_dim);
    // beyond 2^31 turns a position a double has no fraction worth the name
    if (!(f >= 0.0 && f < 1.3e10 && f / (scaling ? factor : 1.0) < 1.3e10)) return DSPARK_ERR_ARG;
  }
  dspark::rope_table(rot_dim, base, scaling, factor, original_len, low, high, inv_freq, table);
  return 0;
}

// the sizes of a rotation; dtypes: src fp32 or dst
static int check_rotation(int32_t src_dtype, int32_t dst_dtype, int32_t n_tokens, int32_t n_heads,
                          int32_t n_kv_heads, int32_t head_dim, int32_t rot_start,
                          int32_t rot_dim, float eps, float magnitude) {
  for (int32_t d : {src_dtype, dst_dtype})
    if (d != DSPARK_F32 && d != DSPARK_BF16 && d != DSPARK_F16) return DSPARK_ERR_DTYPE;
  if (src_dtype != DSPARK_F32 && src_dtype != dst_dtype) return DSPARK_ERR_DTYPE;
  if (n_tokens < 0 || n_heads < 0 || n_kv_heads < 0 || (int64_t)n_heads + n_kv_heads > 65535 ||
      head_dim < 8 || head_dim > DSPARK_MAX_HEAD || head_dim % 8 || rot_start < 0 ||
      rot_start % 8 || rot_dim < 0 || rot_dim % 8 || rot_start + rot_dim > head_dim)
    return DSPARK_ERR_SIZE;
  if (!(eps >= 0.0f && eps <= FLT_MAX) || !(magnitude >= -FLT_MAX && magnitude <= FLT_MAX))
    return DSPARK_ERR_ARG;
  return 0;
}

// a tensor of heads: aligned to 16 bytes, as its strides
static bool aligned_heads(const void* p, int32_t dtype, int64_t token, int64_t head) {
  const int unit = 16 / esize(dtype);
  return aligned(p, 16) && token % unit == 0 && head % unit == 0;
}

int dspark_qk_rotate(const void* q, const void* k, int32_t src_dtype, int64_t q_token_stride,
                     int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                     int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                     const float* q_weight, const float* k_weight, float eps,
                     const int32_t* positions, const uint64_t* table, int32_t rot_start,
                     int32_t rot_dim, int32_t interleaved, float magnitude, void* q_out,
                     int64_t qo_token_stride, int64_t qo_head_stride, void* k_out,
                     int64_t ko_token_stride, int64_t ko_head_stride, int32_t out_dtype,
                     void* stream) {
  const NvtxRange nvtx_range("dspark_qk_rotate");
  if (int e = check_rotation(src_dtype, out_dtype, n_tokens, n_heads, n_kv_heads, head_dim,
                             rot_start, rot_dim, eps, magnitude))
    return e;
  if (n_heads && (q_token_stride < 0 || q_head_stride < 0 || qo_token_stride < 0 ||
                  qo_head_stride < 0))
    return DSPARK_ERR_SIZE;
  if (n_kv_heads && (k_token_stride < 0 || k_head_stride < 0 || ko_token_stride < 0 ||
                     ko_head_stride < 0))
    return DSPARK_ERR_SIZE;
  if (n_tokens == 0 || n_heads + n_kv_heads == 0) return 0;
  if ((n_heads && (!q || !q_out)) || (n_kv_heads && (!k || !k_out)) || !positions ||
      (rot_dim && !table))
    return DSPARK_ERR_NULL;
  if (n_heads && (!aligned_heads(q, src_dtype, q_token_stride, q_head_stride) ||
                  !aligned_heads(q_out, out_dtype, qo_token_stride, qo_head_stride)))
    return DSPARK_ERR_ALIGN;
  if (n_kv_heads && (!aligned_heads(k, src_dtype, k_token_stride, k_head_stride) ||
                     !aligned_heads(k_out, out_dtype, ko_token_stride, ko_head_stride)))
    return DSPARK_ERR_ALIGN;
  if (!aligned(positions, 4) || !aligned_or_null(table, 8) || !aligned_or_null(q_weight, 4) ||
      !aligned_or_null(k_weight, 4))
    return DSPARK_ERR_ALIGN;
  // in place: the same elements at the same places
  if (n_heads && q == q_out && (src_dtype != out_dtype || q_token_stride != qo_token_stride ||
                                q_head_stride != qo_head_stride))
    return DSPARK_ERR_ARG;
  if (n_kv_heads && k == k_out && (src_dtype != out_dtype || k_token_stride != ko_token_stride ||
                                   k_head_stride != ko_head_stride))
    return DSPARK_ERR_ARG;
  if ((n_heads && shares_places<2>({{n_tokens, qo_token_stride}, {n_heads, qo_head_stride}},
                                   head_dim)) ||
      (n_kv_heads && shares_places<2>({{n_tokens, ko_token_stride}, {n_kv_heads, ko_head_stride}},
                                      head_dim)))
    return DSPARK_ERR_SIZE;
  return launch_result(dspark::launch_rotate(
      q, k, nullptr, src_dtype, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
      n_tokens, n_tokens, n_heads, n_kv_heads, head_dim, n_heads ? q_weight : nullptr,
      n_kv_heads ? k_weight : nullptr, eps, positions, table, rot_start, rot_dim,
      interleaved != 0, magnitude, q_out, qo_token_stride, qo_head_stride, k_out, nullptr,
      out_dtype, 0, ko_token_stride, ko_head_stride, 0, 1, nullptr, nullptr,
      static_cast<cudaStream_t>(stream)));
}

int dspark_rotate_write(const void* q, const void* k, const void* v, int32_t src_dtype,
                        int64_t q_token_stride, int64_t q_head_stride, int64_t kv_token_stride,
                        int64_t kv_head_stride, int32_t n_src, int32_t n_heads,
                        int32_t n_kv_heads, int32_t head_dim, const float* q_weight,
                        const float* k_weight, float eps, const int32_t* positions,
                        const uint64_t* table, int32_t rot_start, int32_t rot_dim,
                        int32_t interleaved, float magnitude, void* q_out,
                        int64_t qo_token_stride, int64_t qo_head_stride, void* k_cache,
                        void* v_cache, int32_t cache_dtype, int64_t block_stride,
                        int64_t token_stride, int64_t head_stride, int32_t n_blocks,
                        int32_t page_size, const int32_t* slots, const int32_t* rows,
                        int32_t n_tokens, void* stream) {
  const NvtxRange nvtx_range("dspark_rotate_write");
  if (int e = check_cache(n_blocks, page_size, cache_dtype, block_stride, token_stride,
                          head_stride))
    return e;
  if (int e = check_rotation(src_dtype, cache_dtype, n_tokens, n_heads, n_kv_heads, head_dim,
                             rot_start, rot_dim, eps, magnitude))
    return e;
  if (n_src < 0 || n_kv_heads < 1 || kv_token_stride < 0 || kv_head_stride < 0 ||
      (n_heads && (q_token_stride < 0 || q_head_stride < 0 || qo_token_stride < 0 ||
                   qo_head_stride < 0)))
    return DSPARK_ERR_SIZE;
  if (shares_places<3>({{n_blocks, block_stride}, {page_size, token_stride}, {n_kv_heads, head_stride}},
                       head_dim))
    return DSPARK_ERR_SIZE;
  if (rows && n_heads) return DSPARK_ERR_ARG;
  if (n_tokens == 0 || (n_src == 0 && n_heads == 0)) return 0;
  if (!k || !v || !k_cache || !v_cache || !slots || !positions || (rot_dim && !table) ||
      (n_heads && (!q || !q_out)))
    return DSPARK_ERR_NULL;
  if (!aligned_heads(k, src_dtype, kv_token_stride, kv_head_stride) || !aligned(v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      (n_heads && (!aligned_heads(q, src_dtype, q_token_stride, q_head_stride) ||
                   !aligned_heads(q_out, cache_dtype, qo_token_stride, qo_head_stride))) ||
      !aligned(slots, 4) || !aligned_or_null(rows, 4) || !aligned(positions, 4) ||
      !aligned_or_null(table, 8) || !aligned_or_null(q_weight, 4) ||
      !aligned_or_null(k_weight, 4))
    return DSPARK_ERR_ALIGN;
  if (n_heads && q == q_out && (src_dtype != cache_dtype || q_token_stride != qo_token_stride ||
                                q_head_stride != qo_head_stride))
    return DSPARK_ERR_ARG;
  if (n_heads && shares_places<2>({{n_tokens, qo_token_stride}, {n_heads, qo_head_stride}}, head_dim))
    return DSPARK_ERR_SIZE;
  return launch_result(dspark::launch_rotate(
      q, k, v, src_dtype, q_token_stride, q_head_stride, kv_token_stride, kv_head_stride, n_src,
      n_tokens, n_heads, n_kv_heads, head_dim, n_heads ? q_weight : nullptr, k_weight, eps,
      positions, table, rot_start, rot_dim, interleaved != 0, magnitude, q_out, qo_token_stride,
      qo_head_stride, k_cache, v_cache, cache_dtype, block_stride, token_stride, head_stride,
      n_blocks, page_size, slots, rows, static_cast<cudaStream_t>(stream)));
}

static int check_latent(int32_t latent_dim, int32_t rope_dim) {
  if (latent_dim < 64 || latent_dim > DSPARK_MAX_LATENT || latent_dim % 64 || rope_dim < 0 ||
      rope_dim > DSPARK_MAX_LATENT_ROPE || rope_dim % 8)
    return DSPARK_ERR_SIZE;
  return 0;
}

int dspark_latent_write(const void* c, int64_t c_token_stride, const void* r,
                        int64_t r_token_stride, int32_t src_dtype, int32_t n_src,
                        int32_t latent_dim, int32_t rope_dim, const float* weight, float eps,
                        const int32_t* positions, const uint64_t* table, int32_t interleaved,
                        float magnitude, void* cache, int32_t cache_dtype, int64_t block_stride,
                        int64_t token_stride, int32_t n_blocks, int32_t page_size,
                        const int32_t* slots, const int32_t* rows, int32_t n_tokens,
                        void* stream) {
  const NvtxRange nvtx_range("dspark_latent_write");
  if (int e = check_cache(n_blocks, page_size, cache_dtype, block_stride, token_stride, 0))
    return e;
  if (src_dtype != DSPARK_F32 && src_dtype != cache_dtype) return DSPARK_ERR_DTYPE;
  if (int e = check_latent(latent_dim, rope_dim)) return e;
  if (n_src < 0 || n_tokens < 0 || c_token_stride < 0 || (rope_dim && r_token_stride < 0))
    return DSPARK_ERR_SIZE;
  // rows that overlap would hold either one's elements
  if (shares_places<2>({{n_blocks, block_stride}, {page_size, token_stride}}, latent_dim + rope_dim))
    return DSPARK_ERR_SIZE;
  if (!(eps >= 0.0f && eps <= FLT_MAX) || !(magnitude >= -FLT_MAX && magnitude <= FLT_MAX))
    return DSPARK_ERR_ARG;
  if (n_tokens == 0 || n_src == 0) return 0;
  if (!c || !cache || !slots || !positions || (rope_dim && (!r || !table))) return DSPARK_ERR_NULL;
  if (!aligned_heads(c, src_dtype, c_token_stride, 0) ||
      (rope_dim && !aligned_heads(r, src_dtype, r_token_stride, 0)) || !aligned(cache, 16) ||
      !aligned(slots, 4) || !aligned_or_null(rows, 4) || !aligned(positions, 4) ||
      !aligned_or_null(table, 8) || !aligned_or_null(weight, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_latent_write(
      c, c_token_stride, r, r_token_stride, src_dtype, n_src, latent_dim, rope_dim, weight, eps,
      positions, table, interleaved != 0, magnitude, cache, cache_dtype, block_stride,
      token_stride, n_blocks, page_size, slots, rows, n_tokens,
      static_cast<cudaStream_t>(stream)));
}

static int check_latent_rows(int32_t B, int32_t nodes, int32_t n_heads, int32_t latent_dim) {
  if (B < 0 || B > 65535 || nodes < 1 || nodes > DSPARK_MAX_NODES || n_heads < 1 ||
      n_heads > DSPARK_MAX_LATENT_HEADS)
    return DSPARK_ERR_SIZE;
  return check_latent(latent_dim, 0);
}

int64_t dspark_latent_attention_workspace_bytes(int32_t B, int32_t nodes, int32_t n_heads,
                                                int32_t latent_dim) {
  if (check_latent_rows(B, nodes, n_heads, latent_dim)) return 0;
  return dspark::latent_attention_workspace_bytes(B, nodes, n_heads, latent_dim);
}

int dspark_latent_attention(const void* q, int32_t dtype, int64_t q_req_stride,
                            int64_t q_node_stride, int64_t q_head_stride, int32_t B,
                            int32_t nodes, int32_t n_heads, int32_t latent_dim,
                            int32_t rope_dim, const void* cache, int64_t block_stride,
                            int64_t token_stride, int32_t n_blocks, int32_t page_size,
                            const int32_t* block_table, int64_t table_ld, int32_t max_blocks,
                            const int32_t* ctx_len, const int32_t* n_nodes,
                            const uint64_t* tree_mask, float scale, void* out, float* lse,
                            int32_t* req_status, void* workspace, void* stream) {
  const NvtxRange nvtx_range("dspark_latent_attention");
  if (int e = check_cache(n_blocks, page_size, dtype, block_stride, token_stride, 0)) return e;
  if (int e = check_latent_rows(B, nodes, n_heads, latent_dim)) return e;
  if (int e = check_latent(latent_dim, rope_dim)) return e;
  if (page_size % 8 || token_stride < latent_dim + rope_dim || block_stride < token_stride ||
      token_stride >= (1ll << 39) || block_stride >= (1ll << 39) || max_blocks < 1 ||
      table_ld < max_blocks || (int64_t)max_blocks * page_size > DSPARK_MAX_TOKENS ||
      q_req_stride < 0 || q_node_stride < 0 || q_head_stride < 0)
    return DSPARK_ERR_SIZE;
  // times log2(e) it has to stay finite, or a score of 0 would become NaN
  if (!(scale > -2.3e38f && scale < 2.3e38f)) return DSPARK_ERR_ARG;
  if (B == 0) return 0;
  if (!q || !cache || !block_table || !ctx_len || !n_nodes || !out || !req_status || !workspace)
    return DSPARK_ERR_NULL;
  if (q_req_stride % 8 || q_node_stride % 8 || q_head_stride % 8 || !aligned(q, 16) ||
      !aligned(cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
      !aligned(block_table, 4) || !aligned(ctx_len, 4) || !aligned(n_nodes, 4) ||
      !aligned_or_null(tree_mask, 8) || !aligned_or_null(lse, 4) || !aligned(req_status, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_latent_attention(
      q, dtype, q_req_stride, q_node_stride, q_head_stride, B, nodes, n_heads, latent_dim,
      rope_dim, cache, block_stride, token_stride, n_blocks, page_size, block_table, table_ld,
      max_blocks, ctx_len, n_nodes, tree_mask, scale, out, lse, req_status, workspace,
      static_cast<cudaStream_t>(stream)));
}

int dspark_logits_process(const void* logits, int32_t dtype, int64_t ld, int32_t B, int32_t rows,
                          int32_t V, const int32_t* history, int64_t history_ld,
                          const int32_t* prompt_len, const int32_t* history_len,
                          const int32_t* draft_tokens, int32_t n_drafts,
                          const uint64_t* row_mask, const float* repetition,
                          const float* frequency, const float* presence,
                          const int32_t* bias_ids, const float* bias_values, int32_t max_bias,
                          const int32_t* n_bias, const uint32_t* mask_words, int64_t mask_ld,
                          int32_t n_masks, const int32_t* mask_rows, void* out, int64_t ld_out,
                          int32_t* req_status, void* stream) {
  const NvtxRange nvtx_range("dspark_logits_process");
  if (int e = check_common(dtype, V, ld)) return e;
  if (B < 0 || B > 65535 || rows < 1 || rows > DSPARK_MAX_NODES || ld_out < V || n_drafts < 0 ||
      n_drafts > DSPARK_MAX_NODES || max_bias < 0 || max_bias > 65535 || history_ld < 0 ||
      history_ld >= (1 << 24))
    return DSPARK_ERR_SIZE;
  if (mask_words && (mask_ld < (V + 31) / 32 || n_masks < 1)) return DSPARK_ERR_SIZE;
  if (B == 0) return 0;
  if (!logits || !out || !req_status || (history && !history_len) ||
      (n_drafts > 0 && !draft_tokens) || (max_bias > 0 && (!bias_ids || !bias_values)))
    return DSPARK_ERR_NULL;
  if (out == logits && ld_out != ld) return DSPARK_ERR_ARG;
  const int es = esize(dtype);
  if (!aligned(logits, es) || !aligned(out, es) || !aligned_or_null(history, 4) ||
      !aligned_or_null(prompt_len, 4) || !aligned_or_null(history_len, 4) ||
      !aligned_or_null(draft_tokens, 4) || !aligned_or_null(row_mask, 8) ||
      !aligned_or_null(repetition, 4) || !aligned_or_null(frequency, 4) ||
      !aligned_or_null(presence, 4) || !aligned_or_null(bias_ids, 4) ||
      !aligned_or_null(bias_values, 4) || !aligned_or_null(n_bias, 4) ||
      !aligned_or_null(mask_words, 4) || !aligned_or_null(mask_rows, 4) ||
      !aligned(req_status, 4))
    return DSPARK_ERR_ALIGN;
  return launch_result(dspark::launch_logits_process(
      logits, dtype, ld, B, rows, V, history, history_ld, prompt_len, history_len, draft_tokens,
      n_drafts, row_mask, repetition, frequency, presence, bias_ids, bias_values, max_bias, n_bias,
      mask_words, mask_ld, n_masks, mask_rows, out, ld_out, req_status,
      static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
