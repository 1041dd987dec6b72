// rs_expert_tc_bf16.cu -- the experts' tensor-core products for __nv_bfloat16.
#include "rs_expert_tc_launch.cuh"

template rs_status rsx::tc_ragged_rows<__nv_bfloat16>(const TcOperand<__nv_bfloat16>&, const TcOperand<__nv_bfloat16>&, TcArgs<__nv_bfloat16>, cudaStream_t);
template rs_status rsx::tc_ragged_reduce<__nv_bfloat16>(const TcOperand<__nv_bfloat16>&, const TcOperand<__nv_bfloat16>&, TcArgs<__nv_bfloat16>, cudaStream_t);
