// ida_vec.cuh -- 16-byte vectors of fp32 or bf16 elements, and what the entry points of the
// selective mixer and of the pre-norm share on the host side.
#pragma once

#include <string>

#include "ida_common.cuh"

namespace ida {

// 16 bytes of elements of type E: n elements, unpacked to and packed from fp32.
template <typename E>
struct Vec16;

template <>
struct Vec16<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// log(1 + e^z) without overflow; its derivative is 1 / (1 + e^-z).
__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// The rate e^a_log of a head, 2e38 at most: finite, 1 / ln 2 times it too, so that a step of 0 decays
// nothing.  (At 2e38 a step of 1e-36 decays to 0 already.)
__device__ __forceinline__ float scan_rate(float a_log) {
    const float r = expf(a_log);
    return r > 2e38f ? 2e38f : r;
}

// Programmatic dependent launches (launch_dependent): wait for the launch before in the stream, and let
// the one behind take its place on the SMs.
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependent_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- host side ---------------------------------------------------------------------------

ida_status fail_with(ida_status s, const std::string &why);
ida_status check_call(int d, int R, int M, int W, int dtype, int flags, int *num_sms, std::string &why);

inline bool misaligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Rows of a call's tensor in memory: `rows` of w bytes, ld bytes apart.
struct Rows {
    const char *name;
    const void *p;
    long long ld, w, rows;
};
inline Rows rows_of(const char *name, const void *p, long long ld, long long w, long long rows, int dtype) {
    const long long es = dtype == IDA_F32 ? 4 : 2;
    return {name, p, ld * es, w * es, rows};
}
inline Rows dense(const char *name, const void *p, size_t bytes) { return {name, p, (long long)bytes, (long long)bytes, 1}; }

// Whether two share a byte (slices of the same wider rows do not; rows at two strides whose ranges meet count
// as sharing).
inline bool overlap(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.w < 1 || b.w < 1) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    if (pa >= pb + (uintptr_t)((b.rows - 1) * b.ld + b.w) || pb >= pa + (uintptr_t)((a.rows - 1) * a.ld + a.w)) return false;
    if (a.ld != b.ld || (a.rows == 1 && b.rows == 1)) return true;
    const long long by = (long long)(pb - pa), off = (by % a.ld + a.ld) % a.ld;
    return off < a.w || off + b.w > a.ld;
}

// Outputs share no byte with inputs or one another.
template <int NO, int NI>
ida_status check_overlaps(const Rows (&out)[NO], const Rows (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int k = 0; k < NI; ++k)
            if (overlap(out[i], in[k])) return fail_with(IDA_ERR_ARG, std::string(out[i].name) + " must not overlap " + in[k].name);
        for (int k = i + 1; k < NO; ++k)
            if (overlap(out[i], out[k])) return fail_with(IDA_ERR_ARG, std::string(out[i].name) + " must not overlap " + out[k].name);
    }
    return IDA_OK;
}

// Device set-up of a call whose own arguments have been checked: the number of SMs, and any
// pending device error.
inline ida_status device_ready(int *num_sms, std::string &why) {
    return check_call(8, 8, 1, 1, IDA_F32, 0, num_sms, why);
}

// Head layout of the selective mixer: H heads of d channels, G groups of M state channels.
inline ida_status check_ssm(int H, int d, int G, int M, int dtype) {
    if (d < 1 || M < 1 || G < 1) return fail_with(IDA_ERR_ARG, "d, G and M must be >= 1");
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if (d < 8 || d > 256 || (d % 8) || M < 8 || M > 128 || (M % 8))
        return fail_with(IDA_ERR_UNSUPPORTED, "supported: 8 <= d <= 256 and 8 <= M <= 128, multiples of 8");
    if (H % G) return fail_with(IDA_ERR_ARG, "G must divide H");
    if (H > (1 << 16)) return fail_with(IDA_ERR_UNSUPPORTED, "H above 2^16");
    return IDA_OK;
}

// A launch that may start while the one before it in the stream ends; its kernel waits (dependent_wait)
// before it touches memory.
template <typename... K, typename... A>
cudaError_t launch_dependent(void (*kernel)(K...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, K(args)...);
}
// The attribute that dynamic shared memory above 48 KB needs.
template <typename F>
cudaError_t allow_smem(F *kernel, size_t bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
inline ida_status launched(const char *what) {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
}

}  // namespace ida
