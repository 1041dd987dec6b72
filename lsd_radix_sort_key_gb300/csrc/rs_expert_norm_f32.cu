// rs_expert_norm_f32.cu -- the norms around an expert block for float.
#include "rs_expert_norm_launch.cuh"

template rs_status rsx::norm_forward<float>(const NormArgs<float>&, bool, cudaStream_t);
template rs_status rsx::norm_gradient<float>(const NormArgs<float>&, bool, uint32_t, cudaStream_t);
