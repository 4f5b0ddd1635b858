// ida_ssm.cuh -- what the kernels of the selective scan share.
//
// Per row b and head h (group g = h / (H / G)), with D_t = softplus(dt_t + dt_bias):
//   X_t = a_t X_{t-1} + D_t b_t x_t^T,   a_t = exp(-e^{a_log} D_t),   y_t = X_t^T c_t + D x_t,
// X [M][d] in fp32.
#pragma once

#include "ida_vec.cuh"

namespace ida {

struct ScanArgs {
    const void *x, *b, *c, *dt;
    const float *a_log, *dt_bias, *D, *state_in;
    void *y;
    float *final_state;
    int B, H, N, d, G, M;
    long long ldx, ldb, ldc, lddt;
    int seg, segs;      // positions per segment, segments per sequence
    int fine;           // parts of a segment that a first launch takes by themselves (tensor cores)
    int state_segs;     // parts whose last state from zero that launch leaves in seg_state
    float *seg_state;   // [B H][segs fine][M][d]: each part's last state from zero
    float *seg_log;     // [B H][segs fine]: the sum of log a over the part (of log2 a on the tensor cores)
    unsigned *err;
};

struct ScanBwdArgs {
    const void *x, *b, *c, *dt, *dy;
    const float *a_log, *dt_bias, *D;
    void *dx, *db, *dc, *ddt;
    float *da_log, *ddt_bias, *dD;
    int B, H, N, d, G, M;
    long long ldx, ldb, ldc, lddt, lddx, lddb, lddc, ldddt;
    int chunk, chunks;
    float *state0;   // [B H][chunks][M][d]: the state before each chunk
    float *adj;      // [B H][chunks][M][d]: a Z of the first position behind each chunk
    float *chunk_log;  // [B H][chunks]: the sum of log2 a over the chunk
    float *db_head, *dc_head;  // [B][N][H][M] per head, or NULL where nothing is left to sum
    float *part;     // [B H][chunks][4] ([4][4] on the tensor cores): the chunk's parts of da_log, ddt_bias, dD
    float *kept;     // [B H][chunks][chunk / 8][M][d]: the states behind its groups of 8 positions (CUDA cores)
    unsigned *err;
};

// Two fp32 in one 64-bit register for the packed fp32x2 instructions (each lane rounded like
// the scalar instruction).
typedef unsigned long long ssm_f2;
__device__ __forceinline__ ssm_f2 ssm_pack(float lo, float hi) {
    ssm_f2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void ssm_unpack(ssm_f2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ ssm_f2 ssm_fma(ssm_f2 a, ssm_f2 b, ssm_f2 c) {
    ssm_f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ ssm_f2 ssm_mul(ssm_f2 a, ssm_f2 b) {
    ssm_f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

}  // namespace ida
