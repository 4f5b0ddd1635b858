// ida_skinny.cuh -- products of a few rows (ida_skinny.cu).
#pragma once

#include "ida_vec.cuh"

namespace ida {

constexpr int kFewRows = 32;  // rows up to which a call takes them

struct SkinnyArgs {
    const void *x;                  // T rows of K channels, ldx elements apart
    long long ldx;
    const void *w0, *w1;            // [N, K]; w1: the gate's other factor
    void *out, *out_g, *out_u;      // [T, N]; the factors where they are wanted
    const float *sa, *s0, *s1;      // e4m3: scales of x, w0 and w1
    float *so;                      // e4m3 gate: output scales
    int T, K, N;
    bool out_f32, weights_ready;    // weights_ready: nothing in flight writes them when the kernel may start
};

ida_status skinny_product(const SkinnyArgs &a, bool e4m3, int num_sms, cudaStream_t st);  // out = x w0^T
ida_status skinny_gate(const SkinnyArgs &a, bool e4m3, cudaStream_t st);                  // out = silu(x w0^T) (x w1^T)

}  // namespace ida
