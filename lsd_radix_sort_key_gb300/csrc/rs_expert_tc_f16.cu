// rs_expert_tc_f16.cu -- the experts' tensor-core products for __half.
#include "rs_expert_tc_launch.cuh"

template rs_status rsx::tc_ragged_rows<__half>(const TcOperand<__half>&, const TcOperand<__half>&, TcArgs<__half>, cudaStream_t);
template rs_status rsx::tc_ragged_reduce<__half>(const TcOperand<__half>&, const TcOperand<__half>&, TcArgs<__half>, cudaStream_t);
