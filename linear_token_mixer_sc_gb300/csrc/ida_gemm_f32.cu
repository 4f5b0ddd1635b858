// ida_gemm_f32.cu -- the feed-forward block's products of fp32 operands, each given as three bf16 parts
// (ida_gemm.cuh).
#include "ida_gemm.cuh"

namespace ida {

ida_status gemm_f32(int a_mn, int b_mn, int epi, GemmArgs &g, int num_sms, cudaStream_t st) {
    // 512 contraction elements are summed in TMEM at a time: 32 steps that round towards zero, by
    // 2^-24 of the sum each, bias it by less than 2^-20 of its size
    g.chunk = 8;
    if (epi == kGate) return gemm_launch<0, 0, kSums, kGate, float>(g, num_sms, st);
    if (epi == kGateBwd) return gemm_launch<0, 1, kSums, kGateBwd, float>(g, num_sms, st);
    if (a_mn) return gemm_launch<1, 1, kSums, kPlain, float>(g, num_sms, st);
    if (b_mn) return gemm_launch<0, 1, kSums, kPlain, float>(g, num_sms, st);
    return gemm_launch<0, 0, kSums, kPlain, float>(g, num_sms, st);
}

}  // namespace ida
