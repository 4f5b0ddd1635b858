// ida_e4m3.cu -- matrix products of e4m3 operands with a scale for each block of 128, the feed-forward
// block's first half in them, and the quantiser that lays such operands out.
//
//   q = x / scale to the nearest e4m3 value, scale = max |x| / 448 over 128 channels of a row (or of 128 rows)
//   out = sum over blocks k of 128 channels  sa[t, k] sb[n / 128, k] sum of a[t, .] b[n, .] over the block
//   h = silu(g) u of two such products, quantised again with a scale for 128 channels of each row
#include "ida_gemm.cuh"
#include "ida_skinny.cuh"

namespace ida {

ida_status gemm_e4m3(int epi, int dtype, GemmArgs &g, int num_sms, cudaStream_t st) {
    g.chunk = 1;  // a block of 128 has scales of its own
    if (epi == kGate) return gemm_launch<0, 0, kE4M3, kGate, __nv_bfloat16>(g, num_sms, st);
    if (dtype == IDA_F32) return gemm_launch<0, 0, kE4M3, kPlain, float>(g, num_sms, st);
    return gemm_launch<0, 0, kE4M3, kPlain, __nv_bfloat16>(g, num_sms, st);
}

// ---- the quantiser -------------------------------------------------------------------------------

struct QuantArgs {
    const void *x;
    uint8_t *q;
    float *scale;
    long long ldx;
    int rows, K;
    Divisor blocks;  // of 128 channels in a row (rows times blocks < 2^30)
};

// 8 channels of a row, as they lie in memory
template <typename E>
struct Eight {
    uint4 v[8 / Vec16<E>::n];
    __device__ __forceinline__ void load(const E *p, bool live) {
#pragma unroll
        for (int i = 0; i < 8 / Vec16<E>::n; ++i) v[i] = live ? __ldcs(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8 / Vec16<E>::n; ++i) Vec16<E>::unpack(v[i], x + i * Vec16<E>::n);
    }
    __device__ __forceinline__ float top() const {
        float x[8], m = 0.f;
        unpack(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
        return m;
    }
    __device__ __forceinline__ uint2 quantised(const Quotient &by) const {
        float x[8];
        unpack(x);
        by.scale_up(x);
        return make_uint2(by.four(x), by.four(x + 4));
    }
};

// A scale for 128 channels of a row: 16 threads of 8 channels each, four such groups a thread.
constexpr int QU = 4;
template <typename E>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantArgs a) {
    dependent_wait();
    const int sub = threadIdx.x & 15, kb = (int)a.blocks.d;
    const int units = a.rows * kb, u0 = blockIdx.x * (16 * QU) + (threadIdx.x >> 4);
    Eight<E> x[QU];
    long long at[QU];
    bool live[QU];
#pragma unroll
    for (int i = 0; i < QU; ++i) {
        const int u = u0 + 16 * i, r = divide(u < units ? u : 0, a.blocks), c = (u - r * kb) * 128 + sub * 8;
        live[i] = u < units && c < a.K;
        at[i] = (long long)r * a.K + c;
        x[i].load(static_cast<const E *>(a.x) + (long long)r * a.ldx + c, live[i]);
    }
#pragma unroll
    for (int i = 0; i < QU; ++i) {
        float top = x[i].top();
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float sc = quant_scale(top);
        const uint2 q = x[i].quantised(Quotient(sc));
        if (live[i]) __stcs(reinterpret_cast<uint2 *>(a.q + at[i]), q);
        if (sub == 0 && u0 + 16 * i < units) a.scale[u0 + 16 * i] = sc;
    }
}

// A scale for a block of 128 x 128, a CTA for each: 16 threads of 8 channels by 32 rows, 4 passes.
template <typename E>
__global__ void __launch_bounds__(512) quant_blocks_kernel(QuantArgs a) {
    __shared__ float red[16];
    dependent_wait();
    const int rb = divide(blockIdx.x, a.blocks), c = (blockIdx.x - rb * (int)a.blocks.d) * 128 + (threadIdx.x & 15) * 8;
    const long long r0 = (long long)rb * 128 + (threadIdx.x >> 4);
    Eight<E> x[4];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].load(static_cast<const E *>(a.x) + (r0 + 32 * i) * a.ldx + c, r0 + 32 * i < a.rows && c < a.K);
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, x[i].top());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, red[i]);
    const float sc = quant_scale(top);
    const Quotient by(sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long r = r0 + 32 * i;
        const uint2 q = x[i].quantised(by);
        if (r < a.rows && c < a.K) *reinterpret_cast<uint2 *>(a.q + r * a.K + c) = q;
    }
    if (threadIdx.x == 0) a.scale[blockIdx.x] = sc;
}

template <typename E>
static cudaError_t launch_quant(const QuantArgs &a, int block_rows, cudaStream_t st) {
    const long long kb = a.blocks.d;
    if (block_rows == 128)
        return launch_dependent(quant_blocks_kernel<E>, dim3((unsigned)(((long long)a.rows + 127) / 128 * kb)), dim3(512), 0, st, a);
    return launch_dependent(quant_rows_kernel<E>, dim3((unsigned)((a.rows * kb + 16 * QU - 1) / (16 * QU))), dim3(256), 0, st, a);
}

// Sizes of a product: `rows` by N, contracted over K.
static ida_status check_product(int rows, int K, int N, const char *k, const char *n) {
    if (rows < 0) return fail_with(IDA_ERR_ARG, "rows must be >= 0");
    if (K < 1 || N < 1) return fail_with(IDA_ERR_ARG, std::string(k) + " and " + n + " must be >= 1");
    if (K > 65536 || N > 65536 || (K % 16)) return fail_with(IDA_ERR_UNSUPPORTED, std::string("supported: ") + k + " and " + n + " up to 65536, " + k + " % 16 == 0");
    if (rows > (1 << 28) || (long long)rows * (K > N ? K : N) > (1LL << 36))
        return fail_with(IDA_ERR_UNSUPPORTED, std::string("rows above 2^28, or rows times ") + k + " or " + n + " above 2^36");
    return IDA_OK;
}

template <int N>
static ida_status check_pointers(const void *const (&ptrs)[N]) {
    for (const void *p : ptrs) {
        if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
        if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
    }
    return IDA_OK;
}

static long long blocks_of(long long n) { return (n + 127) / 128; }

}  // namespace ida

extern "C" {

ida_status ida_quant_e4m3(const void *x, void *q, float *scale, int rows, int K, int block_rows, long long ldx, int dtype,
                          ida_stream_t stream) {
    using namespace ida;
    if (rows < 0) return fail_with(IDA_ERR_ARG, "rows must be >= 0");
    if (K < 1) return fail_with(IDA_ERR_ARG, "K must be >= 1");
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if (block_rows != 1 && block_rows != 128) return fail_with(IDA_ERR_UNSUPPORTED, "supported: block_rows 1 or 128");
    if (K > 65536 || (K % 16)) return fail_with(IDA_ERR_UNSUPPORTED, "supported: K a multiple of 16 up to 65536");
    if (rows > (1 << 28) || (long long)rows * K > (1LL << 36)) return fail_with(IDA_ERR_UNSUPPORTED, "rows above 2^28, or rows times K above 2^36");
    if (rows > 1 && ldx < K) return fail_with(IDA_ERR_ARG, "ldx must be at least K");
    if (rows > 1 && ((ldx % 8) || ldx > (1LL << 32))) return fail_with(IDA_ERR_UNSUPPORTED, "ldx must be a multiple of 8 up to 2^32");
    if (rows == 0) return IDA_OK;
    if (rows == 1) ldx = K;
    const void *ptrs[] = {x, q, scale};
    ida_status s = check_pointers(ptrs);
    if (s != IDA_OK) return s;
    const size_t scales = (size_t)(block_rows == 1 ? rows : blocks_of(rows)) * blocks_of(K) * 4;
    const Rows outs[] = {dense("q", q, (size_t)rows * K), dense("scale", scale, scales)};
    const Rows ins[] = {rows_of("x", x, ldx, K, rows, dtype)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    const QuantArgs a = {x, static_cast<uint8_t *>(q), scale, ldx, rows, K, divisor((unsigned)blocks_of(K))};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == IDA_F32 ? launch_quant<float>(a, block_rows, st) : launch_quant<__nv_bfloat16>(a, block_rows, st);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("quantiser launch: ") + cudaGetErrorString(e));
    return launched("quantiser");
}

ida_status ida_gemm_e4m3(const void *a, const float *a_scale, const void *b, const float *b_scale, void *out, int rows, int K, int N,
                         int dtype, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_product(rows, K, N, "K", "N");
    if (s != IDA_OK) return s;
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if (N % 8) return fail_with(IDA_ERR_UNSUPPORTED, "supported: N % 8 == 0");
    if (rows == 0) return IDA_OK;
    const void *ptrs[] = {a, a_scale, b, b_scale, out};
    s = check_pointers(ptrs);
    if (s != IDA_OK) return s;
    const size_t kb = (size_t)blocks_of(K), es = dtype == IDA_BF16 ? 2 : 4;
    const Rows outs[] = {dense("out", out, (size_t)rows * N * es)};
    const Rows ins[] = {dense("a", a, (size_t)rows * K), dense("a_scale", a_scale, rows * kb * 4), dense("b", b, (size_t)N * K),
                        dense("b_scale", b_scale, (size_t)blocks_of(N) * kb * 4)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    if (rows <= kFewRows) {
        SkinnyArgs k = {a, K, b, nullptr, out, nullptr, a_scale, b_scale, nullptr, nullptr, rows, K, N, dtype == IDA_F32, false};
        return skinny_product(k, kFewE4M3, num_sms, reinterpret_cast<cudaStream_t>(stream));
    }
    GemmArgs g = {};
    s = device_error_word(&g.err, why);
    if (s != IDA_OK) return fail_with(s, why);
    g.problems = g.segs = 1;
    g.M[0] = rows, g.N[0] = N;
    g.kblocks = (int)kb;
    g.sa = a_scale, g.sb[0] = b_scale;
    g.out[0] = out;
    s = gemm_map(&g.a[0], a, kMapBytes, K, rows, 1, K, 128, 128);
    if (s == IDA_OK) s = gemm_map(&g.b[0], b, kMapBytes, K, N, 1, K, 128, 128);
    if (s == IDA_OK) s = gemm_map(&g.o[0], out, dtype == IDA_BF16 ? kMapBf16 : kMapF32, N, rows, 1, N, dtype == IDA_BF16 ? 64 : 32, 32);
    if (s == IDA_OK) s = gemm_e4m3(kPlain, dtype, g, num_sms, reinterpret_cast<cudaStream_t>(stream));
    return s;
}

ida_status ida_glu_e4m3(const void *a, const float *a_scale, const void *w_gate, const float *gate_scale, const void *w_up,
                        const float *up_scale, void *q, float *scale, int rows, int D, int F, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_product(rows, D, F, "D", "F");
    if (s != IDA_OK) return s;
    if (F % 16) return fail_with(IDA_ERR_UNSUPPORTED, "supported: F % 16 == 0");
    if (rows == 0) return IDA_OK;
    const void *ptrs[] = {a, a_scale, w_gate, gate_scale, w_up, up_scale, q, scale};
    s = check_pointers(ptrs);
    if (s != IDA_OK) return s;
    const size_t kb = (size_t)blocks_of(D), fb = (size_t)blocks_of(F);
    const Rows outs[] = {dense("q", q, (size_t)rows * F), dense("scale", scale, rows * fb * 4)};
    const Rows ins[] = {dense("a", a, (size_t)rows * D), dense("a_scale", a_scale, rows * kb * 4), dense("w_gate", w_gate, (size_t)F * D),
                        dense("gate_scale", gate_scale, fb * kb * 4), dense("w_up", w_up, (size_t)F * D), dense("up_scale", up_scale, fb * kb * 4)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    if (rows <= kFewRows) {
        SkinnyArgs k = {a, D, w_gate, w_up, q, nullptr, a_scale, gate_scale, up_scale, scale, rows, D, F, false, false};
        return skinny_gate(k, kFewE4M3, reinterpret_cast<cudaStream_t>(stream));
    }
    GemmArgs g = {};
    s = device_error_word(&g.err, why);
    if (s != IDA_OK) return fail_with(s, why);
    g.problems = g.segs = 1;
    g.M[0] = rows, g.N[0] = F;
    g.kblocks = (int)kb;
    g.sa = a_scale, g.sb[0] = gate_scale, g.sb[1] = up_scale;
    g.so = scale;
    s = gemm_map(&g.a[0], a, kMapBytes, D, rows, 1, D, 128, 128);
    if (s == IDA_OK) s = gemm_map(&g.b[0], w_gate, kMapBytes, D, F, 1, D, 128, 128);
    if (s == IDA_OK) s = gemm_map(&g.b[1], w_up, kMapBytes, D, F, 1, D, 128, 128);
    if (s == IDA_OK) s = gemm_map(&g.o[0], q, kMapBytes, F, rows, 1, F, 64, 32);
    if (s == IDA_OK) s = gemm_e4m3(kGate, IDA_BF16, g, num_sms, reinterpret_cast<cudaStream_t>(stream));
    return s;
}

}  // extern "C"
