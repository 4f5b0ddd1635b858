// ida_gemm_bf16.cu -- the feed-forward block's products of bf16 operands (ida_gemm.cuh).
#include "ida_gemm.cuh"

namespace ida {

ida_status gemm_bf16(int a_mn, int b_mn, int epi, GemmArgs &g, int num_sms, cudaStream_t st) {
    using E = __nv_bfloat16;
    // The gate's and its gradients' contraction is a row's channels, 65536 at most: sums of one sign lose below 2^-11
    // of themselves, about half of that in truth (of 2048 channels 2^-16).
    if (epi == kGate) return gemm_launch<0, 0, kDirect, kGate, E>(g, num_sms, st);
    if (epi == kGateBwd) return gemm_launch<0, 1, kDirect, kGateBwd, E>(g, num_sms, st);
    // The others' may be the rows, without end: 4096 elements are summed in TMEM at a time, 256 steps, below 2^-15.  (It
    // costs no time: gradients of 16384 rows of 768 and 2048 channels 198 us, 197 with whole sums in TMEM; of 2^20
    // rows of 64 and 64 1284 and 1284; the block of 16384 rows of 2048 and 5632 channels 571 and 570.)
    g.chunk = 64;
    if (a_mn) return gemm_launch<1, 1, kSums, kPlain, E>(g, num_sms, st);
    if (b_mn) return gemm_launch<0, 1, kSums, kPlain, E>(g, num_sms, st);
    return gemm_launch<0, 0, kSums, kPlain, E>(g, num_sms, st);
}

}  // namespace ida
