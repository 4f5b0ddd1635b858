// ida_ffn_simt.cuh -- the feed-forward block's fp32 products on the CUDA cores (ida_ffn_simt.cu).
#pragma once

#include "ida_vec.cuh"

namespace ida {

struct SimtArgs {
    const float *a[3], *b[3];      // operands of each problem (kGate: b[1] the other factor; of each half of the contraction: dx)
    long long lda[3], ldb[3];
    float *out[3];                 // kPlain: of each problem; kGate: h, and the factors or NULL; kGateBwd: dg, du
    const float *gate, *up;        // kGateBwd
    int M[3], N[3], K;             // rows, columns, contraction (of each half)
    int problems, halves;
};

// out = a b^T by operand layout (a_mn, b_mn: the contraction is the outer dimension in memory) and epilogue
ida_status ffn_simt(int a_mn, int b_mn, int epi, const SimtArgs &a, cudaStream_t st);

}  // namespace ida
