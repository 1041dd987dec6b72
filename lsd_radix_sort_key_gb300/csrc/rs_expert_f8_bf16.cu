// rs_expert_f8_bf16.cu -- the experts' products in 8 bits with outputs of __nv_bfloat16.
#include "rs_expert_f8_launch.cuh"

template rs_status rsx::f8_product<__nv_bfloat16>(const F8Operands&, const F8Args<__nv_bfloat16>&, cudaStream_t);
