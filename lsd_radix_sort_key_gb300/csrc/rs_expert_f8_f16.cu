// rs_expert_f8_f16.cu -- the experts' products in 8 bits with outputs of __half.
#include "rs_expert_f8_launch.cuh"

template rs_status rsx::f8_product<__half>(const F8Operands&, const F8Args<__half>&, cudaStream_t);
