// ida_ssm_tc.cuh -- what the tensor-core kernels of the selective scan share: tiles with the
// 128-byte swizzle, their descriptors and tensor maps, decays in fixed point.
#pragma once

#include <cuda.h>

#include "ida_ssm.cuh"
#include "tc_sm103.cuh"

namespace ida {

constexpr int SQ = 128;          // positions per chunk
constexpr int SSLAB = SQ * 128;  // bytes of 128 rows of 64 bf16

// Shared-memory descriptor of a 128-byte-swizzled operand whose 64-element rows are 128 bytes
// apart: 1024 bytes between groups of 8 rows; `lbo` between 64-element slabs (MN-major operands).
__device__ __forceinline__ tc::SmemDesc sw_desc(uint32_t addr, uint32_t lbo) {
    return {((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16), (1024u >> 4) | (1u << 14) | (2u << 29)};
}
__device__ __forceinline__ tc::SmemDesc sw_step(tc::SmemDesc d, uint32_t bytes) {
    d.lo += bytes >> 4;
    return d;
}
// byte offset of 16-byte piece `c` of row `r` in such a slab
__device__ __forceinline__ int sw_off(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void mma_f16_t(uint32_t d, uint32_t a_tmem, tc::SmemDesc b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// log2 of decays in 2^-32 fixed point: their sums and differences are exact.  -2^20 stands for all below
// it, 2^-1048576 being 0: a position's is limited to it, and so are sums over more than a chunk (2^11 such
// positions pass 64 bits).
constexpr float kFix = 4294967296.f, kUnfix = 1.f / 4294967296.f;  // 2^32
constexpr long long kFixLeast = -(1ll << 52);

// 2^x of such an x <= 0, to the accuracy of the hardware exponential however long the decay
__device__ __forceinline__ float ex2_fix(long long x) {
    const float frac = (float)(uint32_t)x * kUnfix;
    return ex2(frac) * ex2((float)(int)(x >> 32));
}

// The rate e^a_log log2 e in two floats: an error in it would be the same in every position of a
// head.  (fp64 issues at a small fraction of the fp32 rate on this part: one warp makes the rates,
// a lane each, and no position takes an fp64 product.)
struct Rate2 {
    float hi, lo;
};
__device__ __forceinline__ Rate2 rate2_of(float a_log) {
    const double e = exp((double)a_log), r = (e > 2e38 ? 2e38 : e) * 1.4426950408889634;
    const float hi = (float)r;
    return {hi, (float)(r - (double)hi)};
}
// log2 of exp(-rate delta) in fixed point, from the exact product of the leading parts
__device__ __forceinline__ long long log2_fix(const Rate2 &rate, float delta) {
    const float p = rate.hi * delta, e = fmaf(rate.hi, delta, -p) + rate.lo * delta;
    if (!(p < 1048576.f)) return kFixLeast;
    return -(__float2ll_rn(p * kFix) + __float2ll_rn(e * kFix));
}

// Running sum of log2 a over a chunk by 128 threads (four warps, named barrier `id`), position k of
// it in thread k; returns the inclusive sum, and the chunk's in `all`.
__device__ __forceinline__ long long chunk_sum(const Rate2 &rate, float delta, int k, long long *tot, long long &all, int id = 1) {
    const int lane = k & 31, w = k >> 5;
    long long fx = log2_fix(rate, delta);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, fx, o);
        if (lane >= o) fx += u;
    }
    if (lane == 31) tot[w] = fx;
    named_sync(id, 128);
    const long long t1 = tot[0], t2 = t1 + tot[1], t3 = t2 + tot[2];
    all = t3 + tot[3];
    named_sync(id, 128);  // the totals have been read
    return fx + (w == 0 ? 0 : w == 1 ? t1 : w == 2 ? t2 : t3);
}

// ---- host side ---------------------------------------------------------------------------

// Rows of B x N positions, ld elements apart, of K units of w bf16 channels each, as a tensor map
// (channel, unit, position, row) with boxes of 64 channels of one unit over `rows` positions.  Channels
// behind w and positions behind N are read as zero and not written.
ida_status ssm_map(CUtensorMap *m, const void *p, int B, int N, int K, int w, long long ld, int rows = SQ);

// Each part's last state from zero (from state_in for the first).
ida_status launch_ssm_states(const ScanArgs &a, cudaStream_t st);

// Every chunk's (a.seg positions) last state from zero, with rev the sum sum_t a_first .. a_t c_t dy_t^T
// of the adjoint it passes on; a.x, a.b and their strides then are dy's and c's.
ida_status launch_ssm_chunk_states(const ScanArgs &a, bool rev, cudaStream_t st);

}  // namespace ida
