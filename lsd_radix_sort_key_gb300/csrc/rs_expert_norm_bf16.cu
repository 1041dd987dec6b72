// rs_expert_norm_bf16.cu -- the norms around an expert block for __nv_bfloat16.
#include "rs_expert_norm_launch.cuh"

template rs_status rsx::norm_forward<__nv_bfloat16>(const NormArgs<__nv_bfloat16>&, bool, cudaStream_t);
template rs_status rsx::norm_gradient<__nv_bfloat16>(const NormArgs<__nv_bfloat16>&, bool, uint32_t, cudaStream_t);
