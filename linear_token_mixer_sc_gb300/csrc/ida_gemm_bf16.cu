// ida_gemm_bf16.cu -- the feed-forward block's products of bf16 operands (ida_gemm.cuh).
#include "ida_gemm.cuh"

namespace ida {

ida_status gemm_bf16(int a_mn, int b_mn, int epi, GemmArgs &g, int num_sms, cudaStream_t st) {
    using E = __nv_bfloat16;
    if (epi == kGate) return gemm_launch<0, 0, kDirect, kGate, E>(g, num_sms, st);
    if (epi == kGateBwd) return gemm_launch<0, 1, kDirect, kGateBwd, E>(g, num_sms, st);
    if (a_mn) return gemm_launch<1, 1, kDirect, kPlain, E>(g, num_sms, st);
    if (b_mn) return gemm_launch<0, 1, kDirect, kPlain, E>(g, num_sms, st);
    return gemm_launch<0, 0, kDirect, kPlain, E>(g, num_sms, st);
}

}  // namespace ida
