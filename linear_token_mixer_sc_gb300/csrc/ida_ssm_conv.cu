// ida_ssm_conv.cu -- the short causal convolution in front of the selective scan, with SiLU,
// and its backward pass.
//
// Per row b, position t and channel c (W <= 4 taps, the last one on the current position):
//   p_t = bias + sum_j w[j] x_{t-W+1+j},   out_t = p_t s_t,   s = 1 / (1 + e^-p),
// with the W - 1 raw rows before position 0 taken from a state (or zero) and the last W - 1
// raw rows handed on.  Backwards, with g_t = dout_t s_t (1 + p_t (1 - s_t)):
//   dx_t = sum_j w[j] g_{t+W-1-j},   dw[j] = sum_t g_t x_{t-W+1+j},   dbias = sum_t g_t.
//
// Both are bound by HBM (about ten operations per element read).  A thread owns four
// neighbouring channels and walks a strip of positions with the W - 1 rows before the current
// one in registers, so each row is read once but for the W - 1 rows that two strips share.
#include "ida_vec.cuh"

namespace ida {

template <typename E>
struct Quad;  // 4 neighbouring elements
template <>
struct Quad<float> {
    typedef float4 raw;
    static __device__ __forceinline__ void unpack(const raw &u, float *x) { x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; }
    static __device__ __forceinline__ raw pack(const float *x) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Quad<__nv_bfloat16> {
    typedef uint2 raw;
    static __device__ __forceinline__ void unpack(const raw &u, float *x) {
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ raw pack(const float *x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};

// the W taps of 4 neighbouring channels, tap by tap
template <int W>
__device__ __forceinline__ void load_taps(const float *w, float (&t)[W][4]) {
    float v[4 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(w) + i);
        v[4 * i] = u.x;
        v[4 * i + 1] = u.y;
        v[4 * i + 2] = u.z;
        v[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) t[j][e] = v[e * W + j];
}

struct ConvArgs {
    const void *x;
    const float *w, *bias, *state_in;
    void *out;
    float *final_state;
    int B, N, C;
    long long ldx;
    int strip, strips;  // positions per strip, strips per row
};

template <typename E>
__device__ __forceinline__ float conv_sigmoid(float p);
// bf16: the hardware exponential and reciprocal, 2^-21 off, are far below the output's rounding
template <>
__device__ __forceinline__ float conv_sigmoid<__nv_bfloat16>(float p) {
    return __fdividef(1.f, 1.f + __expf(-p));
}
template <>
__device__ __forceinline__ float conv_sigmoid<float>(float p) {
    return 1.f / (1.f + expf(-p));
}

constexpr int CONV_THREADS = 256;
constexpr int CONV_BATCH = 8;  // rows whose loads a thread issues together

// Four channels a thread: eight would take 156 registers and leave 8 warps on an SM (94 us for
// 16384 rows of 2176 channels in bf16).
template <typename E, int W>
__global__ void __launch_bounds__(CONV_THREADS, 3) conv_kernel(ConvArgs a) {
    using Q = Quad<E>;
    typedef typename Q::raw raw;
    constexpr int H = W > 1 ? W - 1 : 1;
    const int vecs = a.C / 4;
    const long long item = (long long)blockIdx.x * CONV_THREADS + threadIdx.x;
    if (item >= (long long)a.B * a.strips * vecs) return;
    const int v = (int)(item % vecs), strip = (int)(item / vecs % a.strips), b = (int)(item / vecs / a.strips);
    const int c0 = v * 4, t0 = strip * a.strip, t1 = min(a.N, t0 + a.strip);
    const E *x = static_cast<const E *>(a.x) + (size_t)b * a.N * a.ldx + c0;
    E *out = static_cast<E *>(a.out) + (size_t)b * a.N * a.C + c0;
    float w[W][4], h[H][4];  // h: the rows before the current one, oldest first
    load_taps<W>(a.w + (size_t)c0 * W, w);
    const float4 bv = __ldg(reinterpret_cast<const float4 *>(a.bias + c0));
    const float bias[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[j][e] = 0.f;
        if (t >= 0)
            Q::unpack(__ldg(reinterpret_cast<const raw *>(x + (size_t)t * a.ldx)), h[j]);
        else if (a.state_in)
            Quad<float>::unpack(__ldg(reinterpret_cast<const float4 *>(
                                    a.state_in + ((size_t)b * (W - 1) + (t + W - 1)) * a.C + c0)), h[j]);
    }
    for (int tb = t0; tb < t1; tb += CONV_BATCH) {
        raw u[CONV_BATCH];
#pragma unroll
        for (int k = 0; k < CONV_BATCH; ++k)
            if (tb + k < t1) u[k] = __ldg(reinterpret_cast<const raw *>(x + (size_t)(tb + k) * a.ldx));
#pragma unroll
        for (int k = 0; k < CONV_BATCH; ++k) {
            if (tb + k >= t1) break;
            float cur[4], o[4];
            Q::unpack(u[k], cur);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = fmaf(w[W - 1][e], cur[e], bias[e]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][e], h[j][e], p);
                o[e] = p * conv_sigmoid<E>(p);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) h[j][e] = h[j + 1][e];
                if (W > 1) h[H - 1][e] = cur[e];
            }
            __stcs(reinterpret_cast<raw *>(out + (size_t)(tb + k) * a.C), Q::pack(o));
        }
    }
    if (a.final_state && t1 == a.N)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<float4 *>(a.final_state + ((size_t)b * (W - 1) + j) * a.C + c0) = Quad<float>::pack(h[j]);
}

// ---- backward ------------------------------------------------------------------------------

struct ConvBwdArgs {
    const void *x, *dout;
    const float *w, *bias;
    void *dx;
    float *part;  // [gridDim.x][W + 1][C]: sums of dw[0 .. W) and dbias
    int B, N, C;
    long long ldx, lddx;
    int strip, strips;
};

constexpr int CB_STRIPS = 8;  // strips (rows of threads) of a block at a time
constexpr int CB_BATCH = 4;   // rows whose loads a thread issues together

// Block (32 channel quads) x (8 strips), walking the strips of all rows gridDim.x blocks apart with
// its sums in registers.  A thread walks u = t0 .. t1 + W - 2: it forms g_u from the x window, then
// dx of position u - (W - 1) from the last W values of g, so the W - 1 positions behind a strip are
// evaluated twice (their x and dout come from L2).
template <typename E, int W>
__global__ void __launch_bounds__(32 * CB_STRIPS, 2) conv_bwd_kernel(ConvBwdArgs a) {
    using Q = Quad<E>;
    typedef typename Q::raw raw;
    constexpr int H = W > 1 ? W - 1 : 1;
    __shared__ float red[CB_STRIPS][W + 1][32 * 4];
    const int c0 = (blockIdx.y * 32 + threadIdx.x) * 4;
    float dw[W][4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    if (c0 < a.C) {
        float w[W][4];
        load_taps<W>(a.w + (size_t)c0 * W, w);
        const float4 bv = __ldg(reinterpret_cast<const float4 *>(a.bias + c0));
        const float bias[4] = {bv.x, bv.y, bv.z, bv.w};
        for (long long s = (long long)blockIdx.x * CB_STRIPS + threadIdx.y; s < (long long)a.B * a.strips;
             s += (long long)gridDim.x * CB_STRIPS) {
            const int b = (int)(s / a.strips), t0 = (int)(s % a.strips) * a.strip, t1 = min(a.N, t0 + a.strip);
            const E *x = static_cast<const E *>(a.x) + (size_t)b * a.N * a.ldx + c0;
            const E *dout = static_cast<const E *>(a.dout) + (size_t)b * a.N * a.C + c0;
            E *dx = static_cast<E *>(a.dx) + (size_t)b * a.N * a.lddx + c0;
            float h[H][4], g[H][4];  // the x rows and the g before u
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int t = t0 - (W - 1) + j;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = g[j][e] = 0.f;
                if (t >= 0) Q::unpack(*reinterpret_cast<const raw *>(x + (size_t)t * a.ldx), h[j]);
            }
            const int u1 = t1 + W - 1;  // g beyond position N - 1 is zero
            for (int ub = t0; ub < u1; ub += CB_BATCH) {
                raw rx[CB_BATCH], rd[CB_BATCH];
#pragma unroll
                for (int k = 0; k < CB_BATCH; ++k)
                    if (ub + k < u1 && ub + k < a.N) {
                        rx[k] = *reinterpret_cast<const raw *>(x + (size_t)(ub + k) * a.ldx);
                        rd[k] = *reinterpret_cast<const raw *>(dout + (size_t)(ub + k) * a.C);
                    }
#pragma unroll
                for (int k = 0; k < CB_BATCH; ++k) {
                    const int u = ub + k;
                    if (u >= u1) break;
                    float cur[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f}, o[4];
                    if (u < a.N) {
                        Q::unpack(rx[k], cur);
                        Q::unpack(rd[k], d);
                    }
                    const int t = u - (W - 1);
                    const bool inside = u < t1;  // positions behind the strip are another's to sum
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = fmaf(w[W - 1][e], cur[e], bias[e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][e], h[j][e], p);
                        // the hardware exponential and reciprocal: 2^-21 of a term, for both types
                        const float sg = __fdividef(1.f, 1.f + __expf(-p));
                        const float gu = d[e] * sg * fmaf(p, 1.f - sg, 1.f), gs = inside ? gu : 0.f;
                        db[e] += gs;
                        dw[W - 1][e] = fmaf(gs, cur[e], dw[W - 1][e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(gs, h[j][e], dw[j][e]);
                        // g of positions t .. t + W - 1 = u is g[0 ..], gu; w[j] meets g_{t+W-1-j}
                        o[e] = w[0][e] * gu;
#pragma unroll
                        for (int j = 1; j < W; ++j) o[e] = fmaf(w[j][e], g[W - 1 - j][e], o[e]);
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j) {
                            g[j][e] = g[j + 1][e];
                            h[j][e] = h[j + 1][e];
                        }
                        if (W > 1) {
                            g[H - 1][e] = gu;
                            h[H - 1][e] = cur[e];
                        }
                    }
                    if (t >= t0) *reinterpret_cast<raw *>(dx + (size_t)t * a.lddx) = Q::pack(o);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[threadIdx.y][j][threadIdx.x * 4 + e] = dw[j][e];
        red[threadIdx.y][W][threadIdx.x * 4 + e] = db[e];
    }
    __syncthreads();
    for (int i = threadIdx.y * 32 + threadIdx.x; i < (W + 1) * 32 * 4; i += 32 * CB_STRIPS) {
        const int j = i / (32 * 4), k = i % (32 * 4), c = blockIdx.y * 32 * 4 + k;
        if (c >= a.C) continue;
        float v = 0.f;
#pragma unroll
        for (int y = 0; y < CB_STRIPS; ++y) v += red[y][j][k];
        a.part[((size_t)blockIdx.x * (W + 1) + j) * a.C + c] = v;
    }
}

// dw [C][W] and dbias [C] from the blocks' parts, added in block order within 8 interleaved sums.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float *part, float *dw, float *dbias, int blocks,
                                                           int C, int W) {
    __shared__ float s[8][33];
    const int i = blockIdx.x * 32 + threadIdx.x, total = C * (W + 1);
    float v = 0.f;
    if (i < total)
#pragma unroll 8
        for (int r = threadIdx.y; r < blocks; r += 8) v += part[(size_t)r * total + i];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || i >= total) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
    const int j = i / C, c = i % C;
    if (j < W)
        dw[(size_t)c * W + j] = v;
    else
        dbias[c] = v;
}

// Positions per strip and blocks along the strips of the backward pass.  Two blocks an SM hold the
// sums in registers over all their strips; of the strip lengths 8 .. 64 the one whose longest block
// walks the fewest positions (W - 1 of each strip are walked twice).
static int conv_bwd_strip(int B, int N, int C, long long *blocks) {
    const long long cols = (C / 4 + 31) / 32, most = 304 / cols > 0 ? 304 / cols : 1;
    int best = 0;
    long long cost = 0;
    for (int strip = 64; strip >= 8; strip /= 2) {
        const long long strips = (long long)B * ((N + strip - 1) / strip), want = (strips + CB_STRIPS - 1) / CB_STRIPS;
        const long long n = want < most ? want : most, c = (want + n - 1) / n * (strip + 3);
        if (!best || c < cost) {
            best = strip;
            cost = c;
            *blocks = n;
        }
    }
    return best;
}

static ida_status check_conv(int B, int N, int C, long long ldx, int dtype, int W) {
    if (B < 0 || N < 0) return fail_with(IDA_ERR_ARG, "B and N must be >= 0");
    if (C < 1 || W < 1) return fail_with(IDA_ERR_ARG, "C and W must be >= 1");
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if ((C % 8) || C > (1 << 20) || W > 4)
        return fail_with(IDA_ERR_UNSUPPORTED, "supported: C <= 2^20 (a multiple of 8), W <= 4");
    if (ldx < C) return fail_with(IDA_ERR_ARG, "the row stride is below C");
    if (ldx % 8) return fail_with(IDA_ERR_UNSUPPORTED, "the row stride must be a multiple of 8");
    if (ldx > (1LL << 32) || (long long)B * N > (1LL << 28)) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows");
    return IDA_OK;
}

}  // namespace ida

extern "C" {

ida_status ida_ssm_conv(const void *x, const float *conv_w, const float *conv_b, const float *state_in, void *out,
                        float *final_state, int B, int N, int C, long long ldx, int dtype, int W,
                        ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_conv(B, N, C, ldx, dtype, W);
    if (s != IDA_OK) return s;
    const size_t state_bytes = (size_t)B * (W - 1) * C * sizeof(float);
    if (state_bytes == 0) state_in = final_state = nullptr;
    if (B == 0 || (N == 0 && !final_state)) return IDA_OK;
    if (misaligned16(state_in) || misaligned16(final_state))
        return fail_with(IDA_ERR_ARG, "state_in and final_state must be 16-byte aligned");
    if (overlap(state_in, state_bytes, final_state, state_bytes))
        return fail_with(IDA_ERR_ARG, "state_in and final_state must not overlap");
    if (N > 0) {
        const void *ptrs[] = {x, conv_w, conv_b, out};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
    }
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {  // no positions: the state is handed on
        cudaError_t e = state_in ? cudaMemcpyAsync(final_state, state_in, state_bytes, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(final_state, 0, state_bytes, st);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    }
    ConvArgs a = {x, conv_w, conv_b, state_in, out, final_state, B, N, C, ldx, 0, 0};
    const int vecs = C / 4;
    // strips of 32 positions read 3 / 32 of the rows twice (from L2); shorter ones, down to a
    // batch of loads, where 32 would leave SMs with less than 2048 threads
    a.strip = 32;
    while (a.strip > CONV_BATCH && (long long)B * ((N + a.strip - 1) / a.strip) * vecs < 2048LL * num_sms) a.strip /= 2;
    a.strips = (N + a.strip - 1) / a.strip;
    const long long blocks = ((long long)B * a.strips * vecs + CONV_THREADS - 1) / CONV_THREADS;
    if (blocks > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many elements");
    const unsigned grid = (unsigned)blocks;
#define IDA_CONV(E)                                                                  \
    switch (W) {                                                                     \
        case 1: conv_kernel<E, 1><<<grid, CONV_THREADS, 0, st>>>(a); break;          \
        case 2: conv_kernel<E, 2><<<grid, CONV_THREADS, 0, st>>>(a); break;          \
        case 3: conv_kernel<E, 3><<<grid, CONV_THREADS, 0, st>>>(a); break;          \
        default: conv_kernel<E, 4><<<grid, CONV_THREADS, 0, st>>>(a); break;         \
    }
    if (dtype == IDA_F32) {
        IDA_CONV(float)
    } else {
        IDA_CONV(__nv_bfloat16)
    }
#undef IDA_CONV
    return launched("ssm conv");
}

size_t ida_ssm_conv_backward_workspace_bytes(int B, int N, int C, int W) {
    if (B < 1 || N < 1 || C < 8 || (C % 8) || C > (1 << 20) || W < 1 || W > 4 || (long long)B * N > (1LL << 28)) return 0;
    long long blocks;
    ida::conv_bwd_strip(B, N, C, &blocks);
    return (size_t)blocks * (W + 1) * C * sizeof(float);
}

ida_status ida_ssm_conv_backward(const void *x, const void *dout, const float *conv_w, const float *conv_b, void *dx,
                                 float *dconv_w, float *dconv_b, int B, int N, int C, long long ldx, long long lddx,
                                 int dtype, int W, void *workspace, size_t workspace_bytes, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_conv(B, N, C, ldx, dtype, W);
    if (s == IDA_OK) s = check_conv(B, N, C, lddx, dtype, W);
    if (s != IDA_OK) return s;
    if (!dconv_w || !dconv_b) return fail_with(IDA_ERR_ARG, "null gradient pointer");
    const bool work = B > 0 && N > 0;
    if (work) {
        const void *ptrs[] = {x, dout, conv_w, conv_b, dx, workspace};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input, output or workspace pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        if (workspace_bytes < ida_ssm_conv_backward_workspace_bytes(B, N, C, W))
            return fail_with(IDA_ERR_ARG, "workspace is smaller than ida_ssm_conv_backward_workspace_bytes");
    }
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!work) {
        cudaError_t e = cudaMemsetAsync(dconv_w, 0, (size_t)C * W * sizeof(float), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dconv_b, 0, (size_t)C * sizeof(float), st);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    }
    ConvBwdArgs a = {x, dout, conv_w, conv_b, dx, static_cast<float *>(workspace), B, N, C, ldx, lddx, 0, 0};
    long long blocks;
    a.strip = conv_bwd_strip(B, N, C, &blocks);
    a.strips = (N + a.strip - 1) / a.strip;
    const dim3 grid((unsigned)blocks, (unsigned)((C / 4 + 31) / 32)), block(32, CB_STRIPS);
#define IDA_CONV(E)                                                   \
    switch (W) {                                                      \
        case 1: conv_bwd_kernel<E, 1><<<grid, block, 0, st>>>(a); break;  \
        case 2: conv_bwd_kernel<E, 2><<<grid, block, 0, st>>>(a); break;  \
        case 3: conv_bwd_kernel<E, 3><<<grid, block, 0, st>>>(a); break;  \
        default: conv_bwd_kernel<E, 4><<<grid, block, 0, st>>>(a); break; \
    }
    if (dtype == IDA_F32) {
        IDA_CONV(float)
    } else {
        IDA_CONV(__nv_bfloat16)
    }
#undef IDA_CONV
    s = launched("ssm conv backward");
    if (s != IDA_OK) return s;
    conv_bwd_sum_kernel<<<(unsigned)((C * (W + 1) + 31) / 32), dim3(32, 8), 0, st>>>(a.part, dconv_w, dconv_b,
                                                                                    (int)blocks, C, W);
    return launched("ssm conv parameter gradients");
}

}  // extern "C"
