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
    int parts;                     // of the contraction, each with outputs of its own, part_floats behind the ones before
    long long part_floats;
};

// out = a b^T by operand layout (a_mn, b_mn: the contraction is the outer dimension in memory) and epilogue
ida_status ffn_simt(int a_mn, int b_mn, int epi, const SimtArgs &a, cudaStream_t st);

// Parts into which the weights' gradients' contraction over T rows is taken (three products of D by F)
int ffn_simt_parts(long long T, long long D, long long F);
// out[0 .. 2], n floats each, of `parts` such triples one behind the other
ida_status ffn_simt_add(const float *from, float *const (&out)[3], long long n, int parts, cudaStream_t st);

}  // namespace ida
