// bf16-logit instantiations of the post-training losses' kernel for short rows.
#include "gbce_post_short.cuh"

namespace gbce {
template cudaError_t launch_post_short<__nv_bfloat16>(const PostParams &, int, int, cudaStream_t);
}  // namespace gbce
