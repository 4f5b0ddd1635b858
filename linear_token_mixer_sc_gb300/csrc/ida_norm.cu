// ida_norm.cu -- root-mean-square norm of the residual stream, and its backward pass.
//
// The pages embed the token mixer in a pre-norm decoder ("Interdomain Attention: Beyond
// Token-Level Key-Value Memory", German technical summary, "Skalierbare Implementierung",
// "Architektur").  Between two blocks of it, per row of D channels:
//   r = x + residual (rounded to the stream's type and stored),
//   y = r / sqrt(mean r^2 + eps) * w,
// y in the stream's type or in e4m3 with one fp32 scale per group of channels, for a
// projection in 8 bits:  scale = max |y| / 448 over the group (1 for a group of zeros, rounded up
// where it is subnormal),  q = y / scale.  Backwards, with n = r / rms and g = dy w:
//   dx = (g - n mean(g n)) / rms + dres,   dw = sum over rows of dy n.
//
// Every row is read once, held in registers as fp32 through its reductions, and written once.  Forwards HBM
// bounds it (82 % of a copy's rate); backwards it is at 46 % of DRAM and 60 % of the issue rate.  TPR threads share a row (a power of two, several rows per
// block of 256 threads when TPR < 256), each with NV 16-byte vectors TPR vectors apart, so a
// warp's accesses are contiguous.
#include <cuda_fp8.h>

#include "ida_vec.cuh"

namespace ida {

constexpr float kE4M3Max = 448.f, kLeastNormal = 0x1p-126f;

struct NormArgs {
    const void *x, *residual;
    const float *w;
    void *res_out, *out;
    uint8_t *q;
    float *scale;
    int rows, D, group;  // group: 0 no 8-bit output
    float eps;
};

// Sum or maximum over the TPR threads of a row; `red` holds one float per warp of the block.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (TPR > 32) {
        constexpr int WPR = TPR / 32;  // warps of a row
        const int warp = threadIdx.x >> 5;
        __syncthreads();  // `red` is free
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        const float *r = red + warp / WPR * WPR;
        v = r[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) v = MAX ? fmaxf(v, r[i]) : v + r[i];
    }
    return v;
}

template <typename E, int TPR, int NV>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) rmsnorm_kernel(NormArgs a) {
    using V = Vec16<E>;
    constexpr int BT = TPR > 256 ? TPR : 256, RPB = BT / TPR;  // threads and rows of a block
    __shared__ float red[BT / 32];
    const int t = threadIdx.x % TPR, vecs = a.D / V::n;
    const int row = blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = row < a.rows;  // every thread takes part in the reductions
    const size_t base = (size_t)(live ? row : 0) * a.D;
    float r[NV][V::n];
    float ss = 0.f;
    uint4 u[NV], ur[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * TPR;
        u[i] = ur[i] = make_uint4(0, 0, 0, 0);
        if (live && v < vecs) {
            u[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const E *>(a.x) + base) + v);
            if (a.residual) ur[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const E *>(a.residual) + base) + v);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * TPR;
        V::unpack(u[i], r[i]);
        if (a.residual) {
            float s[V::n];
            V::unpack(ur[i], s);
#pragma unroll
            for (int e = 0; e < V::n; ++e) r[i][e] += s[e];
            // the stored stream is what is normalised, so that the backward pass, which reads
            // it, differentiates this function
            const uint4 p = V::pack(r[i]);
            V::unpack(p, r[i]);
            if (a.res_out && live && v < vecs) reinterpret_cast<uint4 *>(static_cast<E *>(a.res_out) + base)[v] = p;
        } else if (a.res_out && live && v < vecs) {
            reinterpret_cast<uint4 *>(static_cast<E *>(a.res_out) + base)[v] = u[i];
        }
#pragma unroll
        for (int e = 0; e < V::n; ++e) ss = fmaf(r[i][e], r[i][e], ss);
    }
    const float inv = 1.f / sqrtf(row_reduce<TPR, false>(ss, red) / (float)a.D + a.eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * TPR;
        if (v < vecs) {
            float w[V::n];
#pragma unroll
            for (int e = 0; e < V::n; e += 4)
                *reinterpret_cast<float4 *>(w + e) = __ldg(reinterpret_cast<const float4 *>(a.w + v * V::n + e));
#pragma unroll
            for (int e = 0; e < V::n; ++e) {
                r[i][e] = r[i][e] * inv * w[e];
                top = fmaxf(top, fabsf(r[i][e]));
            }
            if (a.out && live) __stcs(reinterpret_cast<uint4 *>(static_cast<E *>(a.out) + base) + v, V::pack(r[i]));
        }
    }
    if (a.group == 0) return;
    // one scale per row, or per `group` channels: 32, 64 or 128 of them are 4 .. 32 neighbouring
    // lanes' vectors, since TPR >= 32
    const bool whole = a.group == a.D;
    if (whole) top = row_reduce<TPR, true>(top, red);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * TPR;
        if (!whole) {
            top = 0.f;
            if (v < vecs)
#pragma unroll
                for (int e = 0; e < V::n; ++e) top = fmaxf(top, fabsf(r[i][e]));
            for (int o = a.group / V::n / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        if (!live || v >= vecs) continue;
        float sc = top > 0.f ? top / kE4M3Max : 1.f, up = 1.f;
        if (sc < kLeastNormal) {  // 1 / sc would overflow, and sc may be 0 or 1.5 times too small
            sc = __fdiv_ru(top, kE4M3Max);
            up = 0x1p64f;
#pragma unroll
            for (int e = 0; e < V::n; ++e) r[i][e] *= up;
        }
        const float is = 1.f / (sc * up);
        uint32_t q[V::n / 4];
#pragma unroll
        for (int e = 0; e < V::n; e += 4) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(r[i][e] * is, r[i][e + 1] * is), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(r[i][e + 2] * is, r[i][e + 3] * is), __NV_SATFINITE, __NV_E4M3);
            q[e / 4] = lo | hi << 16;
        }
        uint8_t *dst = a.q + base + (size_t)v * V::n;
        if (V::n == 8)
            __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(q[0], q[V::n / 4 - 1]));
        else
            __stcs(reinterpret_cast<uint32_t *>(dst), q[0]);
        const int c = v * V::n;
        if (c % a.group == 0) a.scale[(size_t)row * (a.D / a.group) + c / a.group] = sc;
    }
}

template <typename E, int TPR, int NV>
static void launch_norm_nv(const NormArgs &a, cudaStream_t st) {
    constexpr int BT = TPR > 256 ? TPR : 256, RPB = BT / TPR;
    rmsnorm_kernel<E, TPR, NV><<<(unsigned)(((long long)a.rows + RPB - 1) / RPB), BT, 0, st>>>(a);
}

template <typename E, int TPR>
static void launch_norm_tpr(const NormArgs &a, int nv, cudaStream_t st) {
    if (nv <= 1)
        launch_norm_nv<E, TPR, 1>(a, st);
    else if (nv <= 2)
        launch_norm_nv<E, TPR, 2>(a, st);
    else if constexpr (TPR == 512 && Vec16<E>::n == 4)  // fp32 rows of more than 4096 channels
        launch_norm_nv<E, TPR, 4>(a, st);
}

template <typename E>
static void launch_norm(const NormArgs &a, int num_sms, cudaStream_t st) {
    const int vecs = a.D / Vec16<E>::n;
    int tpr = 32;
    // two vectors a thread: 16384 rows of 2048 in 41.8 us, with four 43.7, with one 45.4 (e4m3 output)
    while (tpr < 512 && (vecs + tpr - 1) / tpr > 2) tpr *= 2;
    // few rows: spread each over more threads, down to one vector each
    while (tpr < 512 && (long long)a.rows * tpr * 2 <= (long long)num_sms * 512 && vecs > tpr) tpr *= 2;
    const int nv = (vecs + tpr - 1) / tpr;
    switch (tpr) {
        case 32: launch_norm_tpr<E, 32>(a, nv, st); break;
        case 64: launch_norm_tpr<E, 64>(a, nv, st); break;
        case 128: launch_norm_tpr<E, 128>(a, nv, st); break;
        case 256: launch_norm_tpr<E, 256>(a, nv, st); break;
        default: launch_norm_tpr<E, 512>(a, nv, st); break;
    }
}

// ---- backward ------------------------------------------------------------------------------

struct NormBwdArgs {
    const void *r;
    const float *w;
    const void *dy, *dres;
    void *dx;
    float *part;  // [gridDim.x][D]: each block's sum of dy n
    int rows, D;
    float eps;
};

// Persistent: block i takes rows i RB, ... of every gridDim.x RB; its threads own fixed channels,
// so the sums for dw stay in registers until the end and run in a fixed order.  RB rows at a time
// share the two barriers of a reduction and keep RB rows' loads in flight.
template <typename E, int NV, int RB>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(NormBwdArgs a) {
    using V = Vec16<E>;
    __shared__ float red[16][2 * RB];
    dependent_launch();
    const int vecs = a.D / V::n, t = threadIdx.x, nt = blockDim.x, warp = t >> 5, nwarps = nt >> 5;
    float w[NV][V::n], dw[NV][V::n];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * nt;
#pragma unroll
        for (int e = 0; e < V::n; ++e) {
            dw[i][e] = 0.f;
            w[i][e] = v < vecs ? __ldg(a.w + v * V::n + e) : 0.f;
        }
    }
    for (long long row0 = (long long)blockIdx.x * RB; row0 < a.rows; row0 += (long long)gridDim.x * RB) {
        uint4 ur[RB][NV], ud[RB][NV], us[RB][NV];
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = t + i * nt;
                const bool ok = row0 + k < a.rows && v < vecs;
                const size_t at = (size_t)(row0 + k) * vecs + v;
                ur[k][i] = ud[k][i] = us[k][i] = make_uint4(0, 0, 0, 0);
                if (ok) {
                    ur[k][i] = __ldcs(static_cast<const uint4 *>(a.r) + at);
                    ud[k][i] = __ldcs(static_cast<const uint4 *>(a.dy) + at);
                    if (a.dres) us[k][i] = __ldcs(static_cast<const uint4 *>(a.dres) + at);
                }
            }
        float s[2 * RB];
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            float ss = 0.f, sg = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float r[V::n], d[V::n];
                V::unpack(ur[k][i], r);
                V::unpack(ud[k][i], d);
#pragma unroll
                for (int e = 0; e < V::n; ++e) {
                    ss = fmaf(r[e], r[e], ss);
                    sg = fmaf(d[e] * w[i][e], r[e], sg);
                }
            }
            s[2 * k] = warp_sum(ss);
            s[2 * k + 1] = warp_sum(sg);
        }
        __syncthreads();  // the previous rows' sums have been read
        if ((t & 31) == 0)
#pragma unroll
            for (int k = 0; k < 2 * RB; ++k) red[warp][k] = s[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            if (row0 + k >= a.rows) break;
            float ss = 0.f, sg = 0.f;
            for (int j = 0; j < nwarps; ++j) {
                ss += red[j][2 * k];
                sg += red[j][2 * k + 1];
            }
            const float inv = 1.f / sqrtf(ss / (float)a.D + a.eps);
            const float proj = sg / (float)a.D * inv * inv;  // mean(g n) / rms
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = t + i * nt;
                if (v >= vecs) break;
                float r[V::n], d[V::n], o[V::n];
                V::unpack(ur[k][i], r);
                V::unpack(ud[k][i], d);
                V::unpack(us[k][i], o);
#pragma unroll
                for (int e = 0; e < V::n; ++e) {
                    dw[i][e] = fmaf(d[e] * inv, r[e], dw[i][e]);
                    o[e] += inv * (d[e] * w[i][e] - r[e] * proj);
                }
                __stcs(static_cast<uint4 *>(a.dx) + (size_t)(row0 + k) * vecs + v, V::pack(o));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = t + i * nt;
        if (v >= vecs) break;
#pragma unroll
        for (int e = 0; e < V::n; e += 4)
            *reinterpret_cast<float4 *>(a.part + (size_t)blockIdx.x * a.D + v * V::n + e) =
                make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
    }
}

// out[c] = sum over rows of part[row][c], rows in 32 interleaved parts summed in a fixed order.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *part, float *out, int rows, int C) {
    __shared__ float s[32][33];
    dependent_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < C)
#pragma unroll 10
        for (int r = threadIdx.y; r < rows; r += 32) v += __ldcs(part + (size_t)r * C + c);
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(s[threadIdx.x][threadIdx.y]);  // warp y: the 32 parts of column y
    if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < C) out[blockIdx.x * 32 + threadIdx.y] = v;
}

// Blocks of the backward pass: eight an SM, each with its own sums of dw (8 bytes of traffic per channel
// and block).  16384 rows of 768 channels, two rows at a time: 24.6 us; 912 blocks 26.5, 608 blocks 32.1
// (four rows at a time 29.0, 304 blocks 42.7).
constexpr int NORM_BWD_BLOCKS = 1216;
static int norm_bwd_blocks(int rows, int rb) {
    const long long want = ((long long)rows + rb - 1) / rb;
    return want < NORM_BWD_BLOCKS ? (want > 0 ? (int)want : 1) : NORM_BWD_BLOCKS;
}

template <typename E>
static int launch_norm_bwd(const NormBwdArgs &a, cudaStream_t st) {
    const int vecs = a.D / Vec16<E>::n;
    int nt = (vecs + 31) / 32 * 32, blocks;
    if (nt <= 512) {
        blocks = norm_bwd_blocks(a.rows, 2);
        rmsnorm_bwd_kernel<E, 1, 2><<<blocks, nt, 0, st>>>(a);
    } else if (vecs <= 1024) {  // all rows of bf16
        nt = ((vecs + 1) / 2 + 31) / 32 * 32;
        blocks = norm_bwd_blocks(a.rows, 2);
        rmsnorm_bwd_kernel<E, 2, 2><<<blocks, nt, 0, st>>>(a);
    } else {
        nt = ((vecs + 3) / 4 + 31) / 32 * 32;
        blocks = norm_bwd_blocks(a.rows, 1);
        if constexpr (Vec16<E>::n == 4) rmsnorm_bwd_kernel<E, 4, 1><<<blocks, nt, 0, st>>>(a);
    }
    return blocks;
}

static ida_status check_norm(int rows, int D, float eps, int dtype) {
    if (rows < 0) return fail_with(IDA_ERR_ARG, "rows must be >= 0");
    if (!(eps >= 0.f) || !(eps < 3.0e38f)) return fail_with(IDA_ERR_ARG, "eps must be finite and >= 0");
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if (D < 8 || D > 8192 || (D % 8)) return fail_with(IDA_ERR_UNSUPPORTED, "supported: 8 <= D <= 8192, D % 8 == 0");
    return IDA_OK;
}

}  // namespace ida

extern "C" {

ida_status ida_rmsnorm(const void *x, const void *residual, const float *w, void *res_out, void *out, void *out_e4m3,
                       float *scale, int rows, int D, int group, float eps, int dtype, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_norm(rows, D, eps, dtype);
    if (s != IDA_OK) return s;
    if (group < 0) return fail_with(IDA_ERR_ARG, "group must be >= 0");
    if (group != 0 && group != D && group != 32 && group != 64 && group != 128)
        return fail_with(IDA_ERR_UNSUPPORTED, "supported groups: 32, 64, 128 or D channels");
    if (group != 0 && D % group) return fail_with(IDA_ERR_UNSUPPORTED, "group must divide D");
    if (rows == 0) return IDA_OK;
    if (!x || !w) return fail_with(IDA_ERR_ARG, "null input pointer");
    if (group != 0 ? !out_e4m3 || !scale : !out) return fail_with(IDA_ERR_ARG, "null output pointer");
    const void *ptrs[] = {x, residual, w, res_out, out, out_e4m3};
    for (const void *p : ptrs)
        if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
    if (misaligned16(scale)) return fail_with(IDA_ERR_ARG, "scale must be 16-byte aligned");
    // in place on x or residual: every thread reads its part of a row before it writes it
    const size_t n = (size_t)rows * D, bytes = n * (dtype == IDA_F32 ? 4 : 2);
    const bool on_x = res_out == x, on_residual = res_out == residual;
    const Rows outs[] = {dense("res_out", res_out, bytes), dense("out", out, bytes), dense("out_e4m3", group ? out_e4m3 : nullptr, n),
                         dense("scale", group ? scale : nullptr, group ? n / group * 4 : 0)};
    const Rows ins[] = {dense("x", on_x ? nullptr : x, bytes), dense("residual", on_residual ? nullptr : residual, bytes),
                        dense("w", w, (size_t)D * 4)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    NormArgs a = {x, residual, w, res_out, out, static_cast<uint8_t *>(out_e4m3), scale, rows, D, group, eps};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == IDA_F32)
        launch_norm<float>(a, num_sms, st);
    else
        launch_norm<__nv_bfloat16>(a, num_sms, st);
    return launched("rmsnorm");
}

size_t ida_rmsnorm_backward_workspace_bytes(int rows, int D) {
    if (rows < 1 || D < 8 || D > 8192 || (D % 8)) return 0;
    return (size_t)ida::norm_bwd_blocks(rows, 1) * D * sizeof(float);
}

ida_status ida_rmsnorm_backward(const void *r, const float *w, const void *dy, const void *dres, void *dx, float *dw,
                                int rows, int D, float eps, int dtype, void *workspace, size_t workspace_bytes,
                                ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_norm(rows, D, eps, dtype);
    if (s != IDA_OK) return s;
    if (!dw || misaligned16(dw)) return fail_with(IDA_ERR_ARG, "dw must be a 16-byte aligned pointer");
    if (rows > 0) {
        const void *ptrs[] = {r, w, dy, dx, workspace};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input, output or workspace pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        if (misaligned16(dres)) return fail_with(IDA_ERR_ARG, "dres must be 16-byte aligned");
        if (workspace_bytes < ida_rmsnorm_backward_workspace_bytes(rows, D))
            return fail_with(IDA_ERR_ARG, "workspace is smaller than ida_rmsnorm_backward_workspace_bytes");
        const size_t bytes = (size_t)rows * D * (dtype == IDA_F32 ? 4 : 2);
        const Rows outs[] = {dense("dx", dx, bytes), dense("dw", dw, (size_t)D * 4),
                             dense("workspace", workspace, ida_rmsnorm_backward_workspace_bytes(rows, D))};
        const Rows ins[] = {dense("r", r, bytes), dense("dy", dx == dy ? nullptr : dy, bytes),
                            dense("dres", dx == dres ? nullptr : dres, bytes), dense("w", w, (size_t)D * 4)};
        s = check_overlaps(outs, ins);
        if (s != IDA_OK) return s;
    }
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)D * sizeof(float), st);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    }
    NormBwdArgs a = {r, w, dy, dres, dx, static_cast<float *>(workspace), rows, D, eps};
    const int blocks = dtype == IDA_F32 ? launch_norm_bwd<float>(a, st) : launch_norm_bwd<__nv_bfloat16>(a, st);
    s = launched("rmsnorm backward");
    if (s != IDA_OK) return s;
    const cudaError_t e = launch_dependent(sum_rows_kernel, dim3((unsigned)((D + 31) / 32)), dim3(32, 32), 0, st, a.part, dw, blocks, D);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("rmsnorm weight gradient launch: ") + cudaGetErrorString(e));
    return launched("rmsnorm weight gradient");
}

}  // extern "C"
