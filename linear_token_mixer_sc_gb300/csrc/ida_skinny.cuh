// ida_skinny.cuh -- products of a few rows (ida_skinny.cu).
#pragma once

#include "ida_vec.cuh"

namespace ida {

// Rows up to which a call takes them: the columns of one matrix instruction.  With 2048 and 5632 channels, in us, here
// and on tcgen05: the block in bf16 of 8 rows 18.9 and 29 (of 16 rows, by two instructions, 29 and 28); in e4m3 the
// product back of 8 rows 4.7 and 11, the gate 10.7 and 12 (of 16 rows 15 and 12: the instruction in 8 bits is put
// together from others on this part).  In fp32, here and by ida_ffn_simt.cu: the block of one row 23.5 and 117, of
// 16 rows 147 and 118.
constexpr int kFewRows = 8;
enum { kFewBf16 = 0, kFewE4M3 = 1, kFewF32 = 2 };

struct SkinnyArgs {
    const void *x;                  // T rows of K channels, ldx elements apart (of a bf16 product two such: h in two parts)
    long long ldx;
    const void *w0, *w1;            // [N, K]; w1: the gate's other factor
    void *out;                      // [T, N]: a product in bf16 or fp32, the gate's in two parts of bf16, fp32 or e4m3
    void *acts;                     // gate: NULL, or [3, T, N]: both factors and their product
    const float *sa, *s0, *s1;      // e4m3: scales of x, w0 and w1
    float *so;                      // e4m3 gate: output scales
    int T, K, N;
    bool out_f32, weights_ready;    // weights_ready: nothing in flight writes them when the kernel may start
};

ida_status skinny_product(const SkinnyArgs &a, int type, int num_sms, cudaStream_t st);  // out = x w0^T
ida_status skinny_gate(const SkinnyArgs &a, int type, cudaStream_t st);                   // out = silu(x w0^T) (x w1^T)

}  // namespace ida
