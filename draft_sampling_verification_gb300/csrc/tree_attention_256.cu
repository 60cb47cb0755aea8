// tree_attention_256.cu -- the attention kernels of tree_attention.cuh for
// head_dim 256.
#define DSPARK_TU 14  // this file's number in the checked build's site codes
#include "tree_attention_wide.cuh"

namespace dspark {
namespace attn {

cudaError_t launch_256(const Params& p, int dtype, int sms, cudaStream_t stream) {
  return dtype == DSPARK_BF16 ? launch_dim<__nv_bfloat16, 256>(p, sms, stream)
                              : launch_dim<__half, 256>(p, sms, stream);
}

DSPARK_STALL_SETTER(256)

}  // namespace attn

DSPARK_CHECK_COLLECTOR(tree_attention_256)

}  // namespace dspark
