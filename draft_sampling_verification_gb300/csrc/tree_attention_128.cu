// tree_attention_128.cu -- the attention kernels of tree_attention.cuh for
// head_dim 128.
#define DSPARK_TU 13  // this file's number in the checked build's site codes
#include "tree_attention_wide.cuh"

namespace dspark {
namespace attn {

cudaError_t launch_128(const Params& p, int dtype, int sms, cudaStream_t stream) {
  return dtype == DSPARK_BF16 ? launch_dim<__nv_bfloat16, 128>(p, sms, stream)
                              : launch_dim<__half, 128>(p, sms, stream);
}

DSPARK_STALL_SETTER(128)

}  // namespace attn

DSPARK_CHECK_COLLECTOR(tree_attention_128)

}  // namespace dspark
