// ida_ssm_step.cu -- one position of the selective mixer: the short convolution of the new row
// with the stored rows before it, then one step of the selective scan, both states in place.
//
//   [x | b | c] = SiLU(bias + sum_j w[j] row_{-(W-1)+j}),  D = softplus(dt + dt_bias),
//   X <- e^{-e^{a_log} D} X + D b x^T,   y = X^T c + D_skip x     per head, X [M][d] in fp32.
//
// Bound by HBM: the state is read and written once, in 16-byte accesses; the rest is small.
// A cluster of CTAs holds the H / G heads that share b and c of one (row, group), so that every
// CTA of it reads the group's stored b and c rows before one of them shifts those rows (each CTA
// arrives on the cluster barrier once its reads are done, and waits before the shift: no second
// launch and no copy of the stored rows).  A thread issues the loads of its head's state before
// the convolution and the next head's before it stores the present one's.
#include <cooperative_groups.h>

#include "ida_vec.cuh"

namespace ida {

namespace cg = cooperative_groups;

// Four CTAs of 128 threads an SM, 8 vectors of a thread in flight.  256 rows of 16 heads of 128 x 64
// (276 MB): 56.9 us; 256 threads and 8 vectors, two CTAs 75.2, three 77.5; 4 vectors, three CTAs 65.6;
// 128 threads and 4 vectors, six CTAs 57.3; 8 vectors, six CTAs 61.3; 16 vectors, three CTAs 63.4.
constexpr int STEP_THREADS = 128;
constexpr int STEP_BATCH = 8;  // 16-byte state vectors a thread holds at a time

struct StepArgs {
    const void *xbc, *dt;
    const float *conv_w, *conv_b, *a_log, *dt_bias, *D;
    float *conv_state, *state;
    void *y;
    int B, H, d, G, M, W;
    long long ldx, lddt;
};

template <typename E>
__device__ __forceinline__ float step_conv(const StepArgs &a, const E *row, float *tail, int c, int C, int W,
                                           float *raw) {
    // tail [W-1][C]; raw receives the new rows of the shifted tail
    float p = a.conv_b[c];
    const float cur = to_float(row[c]);
    for (int j = 0; j < W - 1; ++j) {
        const float v = tail[(size_t)j * C + c];
        p = fmaf(a.conv_w[(size_t)c * W + j], v, p);
        if (j > 0) raw[j - 1] = v;
    }
    p = fmaf(a.conv_w[(size_t)c * W + W - 1], cur, p);
    if (W > 1) raw[W - 2] = cur;
    return p / (1.f + expf(-p));
}

template <typename E>
__global__ void __launch_bounds__(STEP_THREADS, 4) step_kernel(StepArgs a) {
    extern __shared__ __align__(16) float sm[];  // b [M], c [M], x [d], partial y [TY][d]
    cg::cluster_group cluster = cg::this_cluster();
    const int M = a.M, d = a.d, H = a.H, G = a.G, W = a.W, rep = H / G;
    const int C = H * d + 2 * G * M;
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const long long bg = blockIdx.x / cs;
    const int b = (int)(bg / G), g = (int)(bg % G), tid = threadIdx.x;
    float *bs = sm, *cc = bs + M, *xs = cc + M, *part = xs + d;
    const int TX = d / 4, TY = STEP_THREADS / TX;  // vectors of a state row; state rows at a time
    const int tx = tid % TX, ty = tid / TX;
    const bool worker = ty < TY;
    const E *row = static_cast<const E *>(a.xbc) + (size_t)b * a.ldx;
    float *tail = a.conv_state + (size_t)b * (W - 1) * C;

    float4 st[STEP_BATCH];
    const auto load = [&](const float *S, int m0) {
#pragma unroll
        for (int i = 0; i < STEP_BATCH; ++i) {
            const int m = m0 + ty + i * TY;
            if (worker && m < M) st[i] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)m * d) + tx);
        }
    };
    int r = rank;  // head of the group
    if (r < rep) load(a.state + ((size_t)b * H + g * rep + r) * M * d, 0);

    // the group's b and c: every CTA of the cluster evaluates them, CTA 0 shifts their rows.
    // 2 M <= 256 channels: two per thread at most
    float raw[3] = {0.f, 0.f, 0.f};
    float raw2[3] = {0.f, 0.f, 0.f};
    const auto bc_of = [&](int i) { return i < M ? H * d + g * M + i : H * d + G * M + g * M + (i - M); };
    if (tid < 2 * M) bs[tid] = step_conv(a, row, tail, bc_of(tid), C, W, raw);  // c follows b
    if (tid + STEP_THREADS < 2 * M)
        bs[tid + STEP_THREADS] = step_conv(a, row, tail, bc_of(tid + STEP_THREADS), C, W, raw2);
    if (cs > 1) cluster.barrier_arrive();  // the stored b and c rows have been read
    for (; r < rep; r += cs) {
        const int h = g * rep + r;
        float *S = a.state + ((size_t)b * H + h) * M * d;
        for (int i = tid; i < d; i += STEP_THREADS) {  // the head's own channels
            float rx[3];
            const int c = h * d + i;
            xs[i] = step_conv(a, row, tail, c, C, W, rx);
            for (int j = 0; j < W - 1; ++j) tail[(size_t)j * C + c] = rx[j];
        }
        const float delta = softplus(to_float(static_cast<const E *>(a.dt)[(size_t)b * a.lddt + h]) + a.dt_bias[h]);
        const float decay = expf(-scan_rate(a.a_log[h]) * delta);
        __syncthreads();
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (worker) {
            const float4 x4 = reinterpret_cast<const float4 *>(xs)[tx];
            const float x[4] = {delta * x4.x, delta * x4.y, delta * x4.z, delta * x4.w};
            for (int m0 = 0; m0 < M; m0 += STEP_BATCH * TY) {
                if (m0 > 0) load(S, m0);
#pragma unroll
                for (int i = 0; i < STEP_BATCH; ++i) {
                    const int m = m0 + ty + i * TY;
                    if (m >= M) break;
                    const float bm = bs[m], cm = cc[m];
                    float4 v = st[i];
                    v.x = fmaf(decay, v.x, bm * x[0]);
                    v.y = fmaf(decay, v.y, bm * x[1]);
                    v.z = fmaf(decay, v.z, bm * x[2]);
                    v.w = fmaf(decay, v.w, bm * x[3]);
                    y[0] = fmaf(cm, v.x, y[0]);
                    y[1] = fmaf(cm, v.y, y[1]);
                    y[2] = fmaf(cm, v.z, y[2]);
                    y[3] = fmaf(cm, v.w, y[3]);
                    __stcs(reinterpret_cast<float4 *>(S + (size_t)m * d) + tx, v);
                }
            }
            reinterpret_cast<float4 *>(part)[ty * TX + tx] = make_float4(y[0], y[1], y[2], y[3]);
        }
        if (r + cs < rep) load(a.state + ((size_t)b * H + h + cs) * M * d, 0);
        __syncthreads();
        for (int k = tid; k < d; k += STEP_THREADS) {
            float o = a.D[h] * xs[k];
            for (int i = 0; i < TY; ++i) o += part[i * d + k];
            from_float(static_cast<E *>(a.y) + ((size_t)b * H + h) * d + k, o);
        }
    }
    if (cs > 1) cluster.barrier_wait();
    if (rank == 0)
        for (int j = 0; j < W - 1; ++j) {
            if (tid < 2 * M) tail[(size_t)j * C + bc_of(tid)] = raw[j];
            if (tid + STEP_THREADS < 2 * M) tail[(size_t)j * C + bc_of(tid + STEP_THREADS)] = raw2[j];
        }
}

template <typename E>
static ida_status launch_step(const StepArgs &a, cudaStream_t st) {
    const int rep = a.H / a.G;
    int cs = 8;  // the portable cluster limit
    while (cs > rep) cs /= 2;
    const int TY = STEP_THREADS / (a.d / 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.G * cs));
    cfg.blockDim = dim3(STEP_THREADS);
    cfg.dynamicSmemBytes = (size_t)(2 * a.M + a.d + TY * a.d) * sizeof(float);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, step_kernel<E>, a);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail_with(IDA_ERR_CUDA, std::string("ssm step launch: ") + cudaGetErrorString(e));
    }
    return launched("ssm step");
}

}  // namespace ida

extern "C" ida_status ida_ssm_step(const void *xbc, const void *dt, const float *conv_w, const float *conv_b,
                                   const float *a_log, const float *dt_bias, const float *D, float *conv_state,
                                   float *state, void *y, int B, int H, int d, int G, int M, long long ldx,
                                   long long lddt, int dtype, int W, ida_stream_t stream) {
    using namespace ida;
    if (B < 0 || H < 0) return fail_with(IDA_ERR_ARG, "B and H must be >= 0");
    ida_status s = check_ssm(H, d, G, M, dtype);
    if (s != IDA_OK) return s;
    if (W < 1) return fail_with(IDA_ERR_ARG, "W must be >= 1");
    if (W > 4) return fail_with(IDA_ERR_UNSUPPORTED, "supported: W <= 4");
    const long long C = (long long)H * d + 2LL * G * M;
    if (ldx < C || lddt < H) return fail_with(IDA_ERR_ARG, "a row stride is below its row");
    if (ldx % 8) return fail_with(IDA_ERR_UNSUPPORTED, "the row stride of xbc must be a multiple of 8");
    if (ldx > (1LL << 32) || lddt > (1LL << 32) || (long long)B * G > (1LL << 27))
        return fail_with(IDA_ERR_UNSUPPORTED, "B*G above 2^27 or a row stride above 2^32");
    if ((long long)B * H == 0) return IDA_OK;
    const void *ptrs[] = {xbc, conv_w, conv_b, a_log, dt_bias, D, state, y};
    for (const void *p : ptrs) {
        if (!p) return fail_with(IDA_ERR_ARG, "null input, state or output pointer");
        if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
    }
    if (!dt || (reinterpret_cast<uintptr_t>(dt) % (dtype == IDA_F32 ? 4 : 2)))
        return fail_with(IDA_ERR_ARG, "dt must be an aligned pointer");
    if (W > 1 && (!conv_state || misaligned16(conv_state)))
        return fail_with(IDA_ERR_ARG, "conv_state must be a 16-byte aligned pointer");
    const long long w = (long long)H * d;
    const size_t par = (size_t)H * 4;
    const Rows outs[] = {rows_of("y", y, w, w, B, dtype), dense("conv_state", conv_state, (size_t)B * (W - 1) * C * 4),
                         dense("state", state, (size_t)B * H * M * d * 4)};
    const Rows ins[] = {rows_of("xbc", xbc, ldx, C, B, dtype), rows_of("dt", dt, lddt, H, B, dtype),
                        dense("conv_w", conv_w, (size_t)C * W * 4), dense("conv_b", conv_b, (size_t)C * 4), dense("a_log", a_log, par),
                        dense("dt_bias", dt_bias, par), dense("D", D, par)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    StepArgs a = {xbc, dt, conv_w, conv_b, a_log, dt_bias, D, conv_state, state, y, B, H, d, G, M, W, ldx, lddt};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == IDA_F32 ? launch_step<float>(a, st) : launch_step<__nv_bfloat16>(a, st);
}
