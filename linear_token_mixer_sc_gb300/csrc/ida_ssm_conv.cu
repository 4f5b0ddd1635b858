// ida_ssm_conv.cu -- the short causal convolution in front of the selective scan, with SiLU,
// and its backward pass.
//
// Per row b, position t and channel c (W <= 4 taps, the last one on the current position):
//   p_t = bias + sum_j w[j] x_{t-W+1+j},   out_t = p_t s_t,   s = 1 / (1 + e^-p),
// with the W - 1 raw rows before position 0 taken from a state (or zero) and the last W - 1
// raw rows handed on.  Backwards, with g_t = dout_t s_t (1 + p_t (1 - s_t)):
//   dx_t = sum_j w[j] g_{t+W-1-j},   dw[j] = sum_t g_t x_{t-W+1+j},   dbias = sum_t g_t.
//
// Forwards the loads in flight bound it (43 % of DRAM and of the issue rate), backwards instructions (57 %
// of the issue rate, 26 % of DRAM).  A thread owns four neighbouring channels and walks a strip of
// positions with the W - 1 rows before the current one in registers, so each row is read once but for the
// W - 1 rows that two strips share.
#include <type_traits>

#include "ida_ssm.cuh"

namespace ida {

// 2 n neighbouring elements, as n pairs for the packed fp32x2 instructions (the kernels' time is the
// instructions of an element as much as its bytes)
template <typename E, int n>
struct Pairs;
template <int n>
struct Pairs<float, n> {
    typedef typename std::conditional<n == 2, float4, float2>::type raw;
    static __device__ __forceinline__ void unpack(const raw &u, ssm_f2 (&x)[n]) {
#pragma unroll
        for (int i = 0; i < n; ++i) x[i] = ssm_pack((&u.x)[2 * i], (&u.x)[2 * i + 1]);
    }
    static __device__ __forceinline__ raw pack(const ssm_f2 (&x)[n]) {
        raw u;
#pragma unroll
        for (int i = 0; i < n; ++i) ssm_unpack(x[i], (&u.x)[2 * i], (&u.x)[2 * i + 1]);
        return u;
    }
};
template <int n>
struct Pairs<__nv_bfloat16, n> {
    typedef typename std::conditional<n == 2, uint2, uint32_t>::type raw;
    static __device__ __forceinline__ void unpack(const raw &u, ssm_f2 (&x)[n]) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(&u)[i];
            x[i] = ssm_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        }
    }
    static __device__ __forceinline__ raw pack(const ssm_f2 (&x)[n]) {
        raw u;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            float lo, hi;
            ssm_unpack(x[i], lo, hi);
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            reinterpret_cast<uint32_t *>(&u)[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return u;
    }
};

// the W taps of 2 n neighbouring channels, tap by tap
template <int W, int n>
__device__ __forceinline__ void load_taps(const float *w, ssm_f2 (&t)[W][n]) {
    float v[2 * n * W];
#pragma unroll
    for (int i = 0; i < 2 * n * W; i += 2) {
        const float2 u = __ldg(reinterpret_cast<const float2 *>(w + i));
        v[i] = u.x;
        v[i + 1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) t[j][i] = ssm_pack(v[2 * i * W + j], v[(2 * i + 1) * W + j]);
}

// 1 / (1 + e^-p) by the hardware exponential and reciprocal (2^-21 off)
__device__ __forceinline__ ssm_f2 fast_sigmoid(ssm_f2 p) {
    float a, b;
    ssm_unpack(ssm_mul(p, ssm_pack(-1.4426950408889634f, -1.4426950408889634f)), a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    a += 1.f;
    b += 1.f;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return ssm_pack(a, b);
}
// bf16: that is far below the rounding of out and dx.  fp32: expf and a division, in both directions
template <typename E>
__device__ __forceinline__ ssm_f2 conv_sigmoid(ssm_f2 p);
template <>
__device__ __forceinline__ ssm_f2 conv_sigmoid<__nv_bfloat16>(ssm_f2 p) {
    return fast_sigmoid(p);
}
template <>
__device__ __forceinline__ ssm_f2 conv_sigmoid<float>(ssm_f2 p) {
    float a, b;
    ssm_unpack(p, a, b);
    return ssm_pack(1.f / (1.f + expf(-a)), 1.f / (1.f + expf(-b)));
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

constexpr int CONV_THREADS = 256;
constexpr int CONV_BATCH = 4;  // rows whose loads a thread issues together

// Four channels a thread, two pairs.  (16384 rows of 2176 channels in bf16: eight channels in 156
// registers, 8 warps an SM, 94 us; four channels in scalar fp32, 21 instructions an element, 41 us; packed,
// three CTAs an SM and 8 rows at a time 32.7; four CTAs and 4 rows 29.8, and 32.1 with the next rows read
// while the present ones are computed.)
template <typename E, int W>
__global__ void __launch_bounds__(CONV_THREADS, 4) conv_kernel(ConvArgs a) {
    using Q = Pairs<E, 2>;
    typedef typename Q::raw raw;
    constexpr int H = W > 1 ? W - 1 : 1;
    const int vecs = a.C / 4;
    const long long item = (long long)blockIdx.x * CONV_THREADS + threadIdx.x;
    if (item >= (long long)a.B * a.strips * vecs) return;
    const int v = (int)(item % vecs), strip = (int)(item / vecs % a.strips), b = (int)(item / vecs / a.strips);
    const int c0 = v * 4, t0 = strip * a.strip, t1 = min(a.N, t0 + a.strip);
    const E *x = static_cast<const E *>(a.x) + ((size_t)b * a.N + t0) * a.ldx + c0;
    E *out = static_cast<E *>(a.out) + ((size_t)b * a.N + t0) * a.C + c0;
    ssm_f2 w[W][2], h[H][2], bias[2];  // h: the rows before the current one, oldest first
    load_taps<W>(a.w + (size_t)c0 * W, w);
    Pairs<float, 2>::unpack(__ldg(reinterpret_cast<const float4 *>(a.bias + c0)), bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int t = t0 - (W - 1) + j;
        h[j][0] = h[j][1] = 0ull;
        if (t >= 0)
            Q::unpack(__ldg(reinterpret_cast<const raw *>(x - (long long)(W - 1 - j) * a.ldx)), h[j]);
        else if (a.state_in)
            Pairs<float, 2>::unpack(__ldg(reinterpret_cast<const float4 *>(
                                        a.state_in + ((size_t)b * (W - 1) + (t + W - 1)) * a.C + c0)), h[j]);
    }
    const auto step = [&](const raw &u, E *o_at) {
        ssm_f2 cur[2], o[2];
        Q::unpack(u, cur);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ssm_f2 p = ssm_fma(w[W - 1][e], cur[e], bias[e]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) p = ssm_fma(w[j][e], h[j][e], p);
            o[e] = ssm_mul(p, conv_sigmoid<E>(p));
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) h[j][e] = h[j + 1][e];
            if (W > 1) h[H - 1][e] = cur[e];
        }
        __stcs(reinterpret_cast<raw *>(o_at), Q::pack(o));
    };
    int tb = t0;
    for (; tb + CONV_BATCH <= t1; tb += CONV_BATCH, x += CONV_BATCH * a.ldx, out += CONV_BATCH * (long long)a.C) {
        raw u[CONV_BATCH];
#pragma unroll
        for (int k = 0; k < CONV_BATCH; ++k) u[k] = __ldg(reinterpret_cast<const raw *>(x + k * a.ldx));
#pragma unroll
        for (int k = 0; k < CONV_BATCH; ++k) step(u[k], out + k * (long long)a.C);
    }
    for (; tb < t1; ++tb, x += a.ldx, out += a.C) step(__ldg(reinterpret_cast<const raw *>(x)), out);
    if (a.final_state && t1 == a.N)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<float4 *>(a.final_state + ((size_t)b * (W - 1) + j) * a.C + c0) = Pairs<float, 2>::pack(h[j]);
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
constexpr int CN = 4;         // channels of a thread, two pairs

// Block (32 x 4 channels) x (8 strips), walking the strips of all rows gridDim.x blocks apart with its
// sums in registers.  A thread walks u = t0 .. t1 + W - 2: it forms g_u from the x window, then dx of
// position u - (W - 1) from the last W values of g, so the W - 1 positions behind a strip are evaluated
// twice (their x and dout come from L2).  The next rows are read as the present ones are taken: 8 x 2048
// rows of 896 channels in 31.8 us, 35.3 with loads and arithmetic in turn; three CTAs an SM spill, 77 us.
template <typename E, int W>
__global__ void __launch_bounds__(32 * CB_STRIPS, 2) conv_bwd_kernel(ConvBwdArgs a) {
    using Q = Pairs<E, 2>;
    typedef typename Q::raw raw;
    constexpr int H = W > 1 ? W - 1 : 1;
    __shared__ float red[CB_STRIPS][W + 1][32 * CN];
    dependent_launch();
    const int c0 = (blockIdx.y * 32 + threadIdx.x) * CN;
    ssm_f2 dw[W][2], db[2] = {0ull, 0ull};
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][0] = dw[j][1] = 0ull;
    if (c0 < a.C) {
        ssm_f2 w[W][2], bias[2];
        load_taps<W>(a.w + (size_t)c0 * W, w);
        Pairs<float, 2>::unpack(__ldg(reinterpret_cast<const float4 *>(a.bias + c0)), bias);
        const ssm_f2 one = ssm_pack(1.f, 1.f), minus = ssm_pack(-1.f, -1.f);
        for (long long s = (long long)blockIdx.x * CB_STRIPS + threadIdx.y; s < (long long)a.B * a.strips;
             s += (long long)gridDim.x * CB_STRIPS) {
            const int b = (int)(s / a.strips), t0 = (int)(s % a.strips) * a.strip, t1 = min(a.N, t0 + a.strip);
            const size_t row = (size_t)b * a.N + t0;
            const E *x = static_cast<const E *>(a.x) + row * a.ldx + c0;
            const E *dout = static_cast<const E *>(a.dout) + row * a.C + c0;
            E *dx = static_cast<E *>(a.dx) + row * a.lddx + c0;
            ssm_f2 h[H][2], g[H][2];  // the x rows and the g before u
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                h[j][0] = h[j][1] = g[j][0] = g[j][1] = 0ull;
                if (t0 - (W - 1) + j >= 0) Q::unpack(*reinterpret_cast<const raw *>(x - (long long)(W - 1 - j) * a.ldx), h[j]);
            }
            const int n = t1 - t0, left = a.N - t0;  // positions of the strip, and of the row from it on
            raw rx[CB_BATCH], rd[CB_BATCH];  // the next rows, on their way
            const auto read = [&](int k, int u) {  // g beyond the row's end is zero
                rx[k] = rd[k] = raw();
                if (u < n + W - 1 && u < left) {
                    rx[k] = *reinterpret_cast<const raw *>(x + u * a.ldx);
                    rd[k] = *reinterpret_cast<const raw *>(dout + u * (long long)a.C);
                }
            };
#pragma unroll
            for (int k = 0; k < CB_BATCH; ++k) read(k, k);
            for (int ub = 0; ub < n + W - 1; ub += CB_BATCH) {
#pragma unroll
                for (int k = 0; k < CB_BATCH; ++k) {
                    const int u = ub + k;
                    if (u >= n + W - 1) break;
                    ssm_f2 cur[2], d[2], o[2];
                    Q::unpack(rx[k], cur);
                    Q::unpack(rd[k], d);
                    read(k, u + CB_BATCH);
                    const bool inside = u < n;  // positions behind the strip are another's to sum
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ssm_f2 p = ssm_fma(w[W - 1][e], cur[e], bias[e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) p = ssm_fma(w[j][e], h[j][e], p);
                        const ssm_f2 sg = conv_sigmoid<E>(p);
                        const ssm_f2 gu = ssm_mul(ssm_mul(d[e], sg), ssm_fma(p, ssm_fma(sg, minus, one), one));
                        const ssm_f2 gs = inside ? gu : 0ull;
                        db[e] = ssm_fma(gs, one, db[e]);
                        dw[W - 1][e] = ssm_fma(gs, cur[e], dw[W - 1][e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][e] = ssm_fma(gs, h[j][e], dw[j][e]);
                        // g of positions t .. t + W - 1 = u is g[0 ..], gu; w[j] meets g_{t+W-1-j}
                        o[e] = ssm_mul(w[0][e], gu);
#pragma unroll
                        for (int j = 1; j < W; ++j) o[e] = ssm_fma(w[j][e], g[W - 1 - j][e], o[e]);
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
                    if (u >= W - 1) *reinterpret_cast<raw *>(dx + (u - (W - 1)) * a.lddx) = Q::pack(o);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float2 v;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            ssm_unpack(dw[j][e], v.x, v.y);
            *reinterpret_cast<float2 *>(&red[threadIdx.y][j][threadIdx.x * CN + 2 * e]) = v;
        }
        ssm_unpack(db[e], v.x, v.y);
        *reinterpret_cast<float2 *>(&red[threadIdx.y][W][threadIdx.x * CN + 2 * e]) = v;
    }
    __syncthreads();
    for (int i = threadIdx.y * 32 + threadIdx.x; i < (W + 1) * 32 * CN; i += 32 * CB_STRIPS) {
        const int j = i / (32 * CN), k = i % (32 * CN), c = blockIdx.y * 32 * CN + k;
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
    dependent_wait();
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
    const long long cols = (C / CN + 31) / 32, most = 304 / cols > 0 ? 304 / cols : 1;
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
    if (N > 0) {
        const void *ptrs[] = {x, conv_w, conv_b, out};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
    }
    const long long n = (long long)B * N;
    const Rows outs[] = {rows_of("out", out, C, C, n, dtype), dense("final_state", final_state, state_bytes)};
    const Rows ins[] = {rows_of("x", x, ldx, C, n, dtype), dense("conv_w", N > 0 ? conv_w : nullptr, (size_t)C * W * 4),
                        dense("conv_b", N > 0 ? conv_b : nullptr, (size_t)C * 4), dense("state_in", state_in, state_bytes)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
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
    // W - 1 rows of a strip are read twice (from L2), and the last of the passes of four blocks an SM may
    // be short: of the strip lengths up to 64 the one that makes a thread's passes read the fewest rows
    long long cost = 0;
    for (int strip = 64; strip >= CONV_BATCH; strip -= CONV_BATCH) {
        const long long n = ((long long)B * ((N + strip - 1) / strip) * vecs + CONV_THREADS - 1) / CONV_THREADS;
        const long long c = (n + 4 * num_sms - 1) / (4 * num_sms) * (strip + W - 1);
        if (!cost || c < cost) {
            a.strip = strip;
            cost = c;
        }
    }
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
    if (misaligned4(dconv_w) || misaligned4(dconv_b)) return fail_with(IDA_ERR_ARG, "dconv_w and dconv_b must be 4-byte aligned");
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
    const long long n = (long long)B * N;
    const size_t wb = (size_t)C * W * 4, bb = (size_t)C * 4;
    const Rows outs[] = {rows_of("dx", dx, lddx, C, n, dtype), dense("dconv_w", dconv_w, wb), dense("dconv_b", dconv_b, bb),
                         dense("workspace", workspace, ida_ssm_conv_backward_workspace_bytes(B, N, C, W))};
    const Rows ins[] = {rows_of("x", x, ldx, C, n, dtype), rows_of("dout", dout, C, C, n, dtype),
                        dense("conv_w", work ? conv_w : nullptr, wb), dense("conv_b", work ? conv_b : nullptr, bb)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
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
    const dim3 grid((unsigned)blocks, (unsigned)((C / CN + 31) / 32)), block(32, CB_STRIPS);
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
    const cudaError_t e = launch_dependent(conv_bwd_sum_kernel, dim3((unsigned)((C * (W + 1) + 31) / 32)), dim3(32, 8), 0, st,
                                           a.part, dconv_w, dconv_b, (int)blocks, C, W);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm conv parameter gradients launch: ") + cudaGetErrorString(e));
    return launched("ssm conv parameter gradients");
}

}  // extern "C"
