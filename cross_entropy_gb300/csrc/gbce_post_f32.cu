// fp32-logit instantiations of the post-training losses' row kernels.
#include "gbce_post.cuh"

namespace gbce {
template cudaError_t launch_post<float>(const PostParams &, int, int, cudaStream_t);
}  // namespace gbce
