// rs_expert_norm_f16.cu -- the norms around an expert block for __half.
#include "rs_expert_norm_launch.cuh"

template rs_status rsx::norm_forward<__half>(const NormArgs<__half>&, bool, cudaStream_t);
template rs_status rsx::norm_gradient<__half>(const NormArgs<__half>&, bool, uint32_t, cudaStream_t);
