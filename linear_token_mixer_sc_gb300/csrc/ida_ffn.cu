// ida_ffn.cu -- the decoder's gated feed-forward block and its gradients.
//
// The pages embed the token mixer in a Llama-style decoder ("Interdomain Attention: Beyond Token-Level
// Key-Value Memory", German technical summary, "Skalierbare Implementierung", "Architektur"); this is the
// other half of such a layer.  Per row of D channels, with F hidden channels:
//   g = x Wg^T,  u = x Wu^T,  h = silu(g) u,  out = h Wd^T,
// and backwards, with s = 1 / (1 + e^-g):
//   dh = dy Wd,  du = dh g s,  dg = dh u s (1 + g (1 - s)),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h.
// Forwards two products: the first one's tile holds 128 columns of g and the same 128 of u, and its epilogue
// makes h of them.  Backwards three: dh's epilogue reads g and u and writes dg and du, dx is one product
// over both halves of its contraction, and the three weights' gradients are one launch.
// fp32 operands are taken apart into three bf16 parts (x = a + b + c, exactly from 2^-110 on), whose six products down
// to 2^-16 make up fp32's; h, dg and du are rounded to bf16 between the products otherwise.
#include <mutex>

#include "ida_ffn_simt.cuh"
#include "ida_gemm.cuh"
#include "ida_skinny.cuh"

namespace ida {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

ida_status gemm_map(CUtensorMap *m, const void *p, int type, long long inner, long long rows, int parts, long long ld, int box0,
                    int box1) {
    const EncodeFn fn = encode_fn();
    if (!fn) return fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int es = type == kMapBf16 ? 2 : type == kMapF32 ? 4 : 1;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)parts};
    // a single part needs no stride of its own (the rows' stands for it: rows times ld may be too long)
    const cuuint64_t strides[2] = {(cuuint64_t)ld * es, (parts > 1 ? (cuuint64_t)rows : 1) * ld * es};
    const cuuint32_t box[3] = {(cuuint32_t)box0, (cuuint32_t)box1, 1}, one[3] = {1, 1, 1};
    const CUresult r = fn(m, type == kMapBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : type == kMapF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                                                                  : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                          3, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box0 * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? IDA_OK : fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

// ---- three bf16 parts of fp32 ------------------------------------------------------------------

struct SplitArgs {
    const float *src[4];
    __nv_bfloat16 *dst[4];  // [3][rows][cols]
    long long rows[4], ld[4];
    int cols[4];
};

// x = a + b + c: a nearest in bf16 (towards zero where that would overflow), b the rest's nearest, c what is left
__device__ __forceinline__ void parts_of(float x, float &a, float &b, float &c) {
    a = __bfloat162float(__float2bfloat16_rn(x));
    if (fabsf(a) > 3.4e38f) a = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r = x - a;
    b = __bfloat162float(__float2bfloat16_rn(r));
    c = r - b;
}

__global__ void __launch_bounds__(256) split_kernel(SplitArgs a) {
    dependent_launch();
    dependent_wait();
    const int i = blockIdx.y, cols = a.cols[i];
    const long long n = a.rows[i] * cols;
    for (long long e = ((long long)blockIdx.x * 256 + threadIdx.x) * 4; e < n; e += (long long)gridDim.x * 1024) {
        const long long r = e / cols;
        const float4 v = *reinterpret_cast<const float4 *>(a.src[i] + r * a.ld[i] + (e - r * cols));
        const float x[4] = {v.x, v.y, v.z, v.w};
        float p[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) parts_of(x[k], p[0][k], p[1][k], p[2][k]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(p[k][0], p[k][1]), hi = __floats2bfloat162_rn(p[k][2], p[k][3]);
            *reinterpret_cast<uint2 *>(a.dst[i] + k * n + e) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
}

static ida_status launch_split(const SplitArgs &a, int count, int num_sms, cudaStream_t st) {
    long long most = 0;
    for (int i = 0; i < count; ++i) most = a.rows[i] * a.cols[i] > most ? a.rows[i] * a.cols[i] : most;
    const long long want = (most + 1023) / 1024, cap = (long long)num_sms * 8;
    const cudaError_t e = launch_dependent(split_kernel, dim3((unsigned)(want < cap ? want : cap), (unsigned)count), dim3(256), 0, st, a);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ffn split launch: ") + cudaGetErrorString(e));
    return launched("ffn split");
}

// ---- workspaces ----------------------------------------------------------------------------------

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// fp32 products on the CUDA cores: little arithmetic (and backwards no large weights' gradients), or few rows forwards,
// or backwards few channels, whose gradients have few tiles.  In us, there and on the tensor cores, forward and backward:
// 512 rows of 256 and 512 channels 19 + 36 and 30 + 57, 251 of 512 and 1024 (2^27) 34 + 65 and 40 + 71, 1024 of 256 and
// 704 (2^27.5) 40 + 80 and 33 + 64, 1 of 2048 and 5632 backwards 328 and 252, 32 of them 122 + 341 and 164 + 238, 64
// 157 + 363 and 165 + 241.  Backwards by channels, 64 rows: of 512 and 1024 44 and 62, 1024 and 1408 73 and 85, 768 and
// 2048 87 and 89, 1024 and 2048 (2^21) 109 and 102, 1024 and 2816 150 and 119 (the same of 8 rows within 5 %; only
// of 256 and 4096 124 and 97); many rows: 2^22 of 8 and 8 2891 and 31482, 2^18 of 32 and 64 315 and 1938, 2^17 of 128
// and 128 (2^14) 812 and 1129, 2^14 of them 112 and 166, of 128 and 256 209 and 182.
static bool on_cuda_cores(long long rows, long long D, long long F, bool backward) {
    const long long all = rows * D * F;
    return backward ? (all <= (1LL << 27) && D * F <= (1LL << 21)) || D * F <= (1LL << 14) : all <= (1LL << 27) || rows <= 64;
}

// Operands of the products: the caller's own tensors in bf16, their parts in the workspace otherwise.
struct Operand {
    const void *p;
    int parts;
    long long rows, cols, ld;
};

struct FfnSpace {
    size_t h, xs, wg, wu, wd, hs, total;                // forwards
    size_t dgu, dys, dgs, dus, dws;                     // backwards
};

// keep: the caller's acts take h
static FfnSpace ffn_space(long long T, int D, int F, int dtype, bool backward, bool keep) {
    FfnSpace s = {};
    const size_t td = (size_t)T * D, tf = (size_t)T * F, df = (size_t)D * F;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    const size_t es = dtype == IDA_BF16 ? 2 : 4;
    if (!backward && (T <= kFewRows || !keep)) s.h = take(tf * (T <= kFewRows ? 4 : es));  // (few rows' h: two parts)
    if (backward) s.dgu = take(2 * tf * es);
    if (dtype == IDA_F32 && !on_cuda_cores(T, D, F, backward)) {
        s.xs = take(6 * td);
        s.wg = take(6 * df);
        s.wu = take(6 * df);
        s.wd = take(6 * df);
        s.hs = take(6 * tf);
        if (backward) {
            s.dys = take(6 * td);
            s.dgs = take(6 * tf);
            s.dus = take(6 * tf);
        }
    } else if (dtype == IDA_F32 && backward) {
        const int n = ffn_simt_parts(T, D, F);
        if (n > 1) s.dws = take(12 * df * n);
    }
    s.total = off;
    return s;
}

// ---- products ------------------------------------------------------------------------------------

// Boxes of 128 rows x 64 of the contraction, or of 64 x 64 where the contraction is the outer dimension.
static ida_status operand_map(CUtensorMap *m, const Operand &o, int mn) {
    return gemm_map(m, o.p, kMapBf16, o.cols, o.rows, o.parts, o.ld, 64, mn ? 64 : 128);
}
// Boxes of 32 rows and columns of what the gate's gradients read and write
static ida_status box_map(CUtensorMap *m, const void *p, int dtype, long long rows, long long cols) {
    return gemm_map(m, p, dtype == IDA_BF16 ? kMapBf16 : kMapF32, cols, rows, 1, cols, 32, 32);
}

// Passes over the contraction for operands a and b: one in bf16, the six products of parts otherwise, the
// smallest first.
static void add_segments(GemmArgs &g, int dtype, int a, int b) {
    static const unsigned char pa[6] = {0, 2, 1, 0, 1, 0}, pb[6] = {2, 0, 1, 1, 0, 0};
    if (dtype == IDA_BF16) {
        g.seg[g.segs++] = {(unsigned char)a, 0, (unsigned char)b, 0};
        return;
    }
    for (int i = 0; i < 6; ++i) g.seg[g.segs++] = {(unsigned char)a, pa[i], (unsigned char)b, pb[i]};
}

static ida_status run_gemm(int a_mn, int b_mn, int epi, GemmArgs &g, int dtype, int num_sms, cudaStream_t st) {
    std::string why;
    const ida_status s = device_error_word(&g.err, why);
    if (s != IDA_OK) return fail_with(s, why);
    return dtype == IDA_BF16 ? gemm_bf16(a_mn, b_mn, epi, g, num_sms, st) : gemm_f32(a_mn, b_mn, epi, g, num_sms, st);
}

// Rows of which a call takes no more
static bool too_many_rows(int rows, int D, int F) { return rows > (1 << 28) || (long long)rows * (D > F ? D : F) > (1LL << 36); }

// Sizes for which a workspace is wanted
static bool valid_sizes(int rows, int D, int F, int dtype) {
    return rows > 0 && D > 0 && F > 0 && D <= 65536 && F <= 65536 && D % 8 == 0 && F % 8 == 0 && !too_many_rows(rows, D, F) &&
           (dtype == IDA_F32 || dtype == IDA_BF16);
}

static ida_status check_ffn(int rows, int D, int F, long long ldx, int dtype) {
    if (rows < 0) return fail_with(IDA_ERR_ARG, "rows must be >= 0");
    if (D < 1 || F < 1) return fail_with(IDA_ERR_ARG, "D and F must be >= 1");
    if (dtype != IDA_F32 && dtype != IDA_BF16) return fail_with(IDA_ERR_ARG, "dtype must be IDA_F32 or IDA_BF16");
    if (D > 65536 || F > 65536 || (D % 8) || (F % 8))
        return fail_with(IDA_ERR_UNSUPPORTED, "supported: D and F multiples of 8 up to 65536");
    if (too_many_rows(rows, D, F))
        return fail_with(IDA_ERR_UNSUPPORTED, "rows above 2^28, or rows times D or F above 2^36");
    if (rows > 1 && ldx < D) return fail_with(IDA_ERR_ARG, "ldx must be at least D");
    if (rows > 1 && ((ldx % 8) || ldx > (1LL << 32))) return fail_with(IDA_ERR_UNSUPPORTED, "ldx must be a multiple of 8 up to 2^32");
    return IDA_OK;
}

}  // namespace ida

extern "C" {

size_t ida_ffn_workspace_bytes(int rows, int D, int F, int dtype, int keep) {
    return ida::valid_sizes(rows, D, F, dtype) ? ida::ffn_space(rows, D, F, dtype, false, keep != 0).total : 0;
}

size_t ida_ffn_backward_workspace_bytes(int rows, int D, int F, int dtype) {
    return ida::valid_sizes(rows, D, F, dtype) ? ida::ffn_space(rows, D, F, dtype, true, true).total : 0;
}

ida_status ida_ffn(const void *x, const void *w_gate, const void *w_up, const void *w_down, void *out, void *acts, int rows, int D,
                   int F, long long ldx, int dtype, void *workspace, size_t workspace_bytes, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_ffn(rows, D, F, ldx, dtype);
    if (s != IDA_OK) return s;
    if (rows == 0) return IDA_OK;
    if (rows == 1) ldx = D;
    const FfnSpace sp = ffn_space(rows, D, F, dtype, false, acts != nullptr);
    const void *ptrs[] = {x, w_gate, w_up, w_down, out};
    for (const void *p : ptrs) {
        if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
        if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
    }
    if (misaligned16(acts)) return fail_with(IDA_ERR_ARG, "acts must be 16-byte aligned");
    if (sp.total > 0 && (!workspace || misaligned16(workspace)))
        return fail_with(IDA_ERR_ARG, "workspace must be a 16-byte aligned pointer");
    if (workspace_bytes < sp.total) return fail_with(IDA_ERR_ARG, "workspace is smaller than ida_ffn_workspace_bytes");
    const size_t es = dtype == IDA_BF16 ? 2 : 4, td = (size_t)rows * D, tf = (size_t)rows * F, df = (size_t)D * F;
    const Rows outs[] = {dense("out", out, td * es), dense("acts", acts, 3 * tf * es), dense("workspace", sp.total ? workspace : nullptr, sp.total)};
    const Rows ins[] = {rows_of("x", x, ldx, D, rows, dtype), dense("w_gate", w_gate, df * es), dense("w_up", w_up, df * es),
                        dense("w_down", w_down, df * es)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

    char *ws = static_cast<char *>(workspace), *ac = static_cast<char *>(acts);
    void *h = ac ? ac + 2 * tf * es : ws + sp.h;
    const int type = dtype == IDA_BF16 ? kFewBf16 : kFewF32;
    if (rows <= kFewRows) {
        // of few rows h stays in two bf16 parts or fp32, in the workspace
        SkinnyArgs a = {x, ldx, w_gate, w_up, ws + sp.h, acts, nullptr, nullptr, nullptr, nullptr, rows, D, F, true, false};
        s = skinny_gate(a, type, st);
        if (s != IDA_OK) return s;
        SkinnyArgs b = {ws + sp.h, F, w_down, nullptr, out, nullptr, nullptr, nullptr, nullptr, nullptr, rows, F, D, dtype == IDA_F32, true};
        return skinny_product(b, type, num_sms, st);
    }
    if (dtype == IDA_F32 && on_cuda_cores(rows, D, F, false)) {
        float *fh = static_cast<float *>(h), *fa = reinterpret_cast<float *>(ac);
        SimtArgs a = {{static_cast<const float *>(x)}, {static_cast<const float *>(w_gate), static_cast<const float *>(w_up)}, {ldx}, {D},
                      {fh, fa, fa ? fa + tf : nullptr}, nullptr, nullptr, {rows}, {F}, D, 1, 1, 1, 0};
        s = ffn_simt(0, 0, kGate, a, st);
        if (s != IDA_OK) return s;
        SimtArgs b = {{fh}, {static_cast<const float *>(w_down)}, {F}, {F}, {static_cast<float *>(out)}, nullptr, nullptr, {rows}, {D}, F, 1, 1, 1, 0};
        return ffn_simt(0, 0, kPlain, b, st);
    }
    const int parts = dtype == IDA_BF16 ? 1 : 3;
    Operand X = {x, parts, rows, D, ldx}, Wg = {w_gate, parts, F, D, D}, Wu = {w_up, parts, F, D, D}, Wd = {w_down, parts, D, F, F},
            H = {h, parts, rows, F, F};
    if (dtype == IDA_F32) {
        SplitArgs a = {{static_cast<const float *>(x), static_cast<const float *>(w_gate), static_cast<const float *>(w_up),
                        static_cast<const float *>(w_down)},
                       {}, {rows, F, F, D}, {ldx, D, D, F}, {D, D, D, F}};
        const size_t at[4] = {sp.xs, sp.wg, sp.wu, sp.wd};
        for (int i = 0; i < 4; ++i) a.dst[i] = reinterpret_cast<__nv_bfloat16 *>(ws + at[i]);
        s = launch_split(a, 4, num_sms, st);
        if (s != IDA_OK) return s;
        X.p = a.dst[0], Wg.p = a.dst[1], Wu.p = a.dst[2], Wd.p = a.dst[3], H.p = ws + sp.hs;
        X.ld = D;
    }
    GemmArgs g = {};
    g.problems = 1;
    g.M[0] = rows, g.N[0] = F;
    g.kblocks = (D + 63) / 64;
    g.keep = ac != nullptr;
    add_segments(g, dtype, 0, 0);
    s = operand_map(&g.a[0], X, 0);
    if (s == IDA_OK) s = operand_map(&g.b[0], Wg, 0);
    if (s == IDA_OK) s = operand_map(&g.b[1], Wu, 0);
    g.out[0] = h, g.out[1] = ac, g.out[2] = ac ? ac + tf * es : nullptr;
    if (s == IDA_OK) s = run_gemm(0, 0, kGate, g, dtype, num_sms, st);
    if (s != IDA_OK) return s;
    if (dtype == IDA_F32) {
        SplitArgs a = {{static_cast<const float *>(h)}, {reinterpret_cast<__nv_bfloat16 *>(ws + sp.hs)}, {rows}, {F}, {F}};
        s = launch_split(a, 1, num_sms, st);
        if (s != IDA_OK) return s;
    }
    GemmArgs d = {};
    d.problems = d.back = 1;
    d.M[0] = rows, d.N[0] = D;
    d.kblocks = (F + 63) / 64;
    add_segments(d, dtype, 0, 0);
    s = operand_map(&d.a[0], H, 0);
    if (s == IDA_OK) s = operand_map(&d.b[0], Wd, 0);
    d.out[0] = out;
    if (s == IDA_OK) s = run_gemm(0, 0, kPlain, d, dtype, num_sms, st);
    return s;
}

ida_status ida_ffn_backward(const void *x, const void *w_gate, const void *w_up, const void *w_down, const void *acts, const void *dout,
                            void *dx, void *dw_gate, void *dw_up, void *dw_down, int rows, int D, int F, long long ldx, int dtype,
                            void *workspace, size_t workspace_bytes, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_ffn(rows, D, F, ldx, dtype);
    if (s != IDA_OK) return s;
    if (rows == 1) ldx = D;
    const size_t es = dtype == IDA_BF16 ? 2 : 4, td = (size_t)rows * D, tf = (size_t)rows * F, df = (size_t)D * F;
    void *dw[] = {dw_gate, dw_up, dw_down};
    for (const void *p : dw)
        if (!p || misaligned16(p)) return fail_with(IDA_ERR_ARG, "weight gradients must be 16-byte aligned pointers");
    const FfnSpace sp = ffn_space(rows, D, F, dtype, true, true);
    if (rows > 0) {
        const void *ptrs[] = {x, w_gate, w_up, w_down, acts, dout, dx, workspace};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input, output or workspace pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        if (workspace_bytes < sp.total) return fail_with(IDA_ERR_ARG, "workspace is smaller than ida_ffn_backward_workspace_bytes");
    }
    const Rows outs[] = {dense("dx", rows ? dx : nullptr, td * es), dense("dw_gate", dw_gate, df * es), dense("dw_up", dw_up, df * es),
                         dense("dw_down", dw_down, df * es), dense("workspace", rows ? workspace : nullptr, sp.total)};
    const Rows ins[] = {rows_of("x", rows ? x : nullptr, ldx, D, rows, dtype), dense("w_gate", w_gate, df * es),
                        dense("w_up", w_up, df * es), dense("w_down", w_down, df * es),
                        dense("acts", rows ? acts : nullptr, 3 * tf * es), dense("dout", rows ? dout : nullptr, td * es)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        for (void *p : dw) {
            const cudaError_t e = cudaMemsetAsync(p, 0, df * es, st);
            if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
        }
        return IDA_OK;
    }
    char *ws = static_cast<char *>(workspace);
    const char *ac = static_cast<const char *>(acts);
    char *dg = ws + sp.dgu, *du = dg + tf * es;
    if (dtype == IDA_F32 && on_cuda_cores(rows, D, F, true)) {
        const float *fx = static_cast<const float *>(x), *fy = static_cast<const float *>(dout), *fa = reinterpret_cast<const float *>(ac);
        float *fg = reinterpret_cast<float *>(dg), *fu = reinterpret_cast<float *>(du);
        SimtArgs a = {{fy}, {static_cast<const float *>(w_down)}, {D}, {F}, {fg, fu}, fa, fa + tf, {rows}, {F}, D, 1, 1, 1, 0};
        s = ffn_simt(0, 1, kGateBwd, a, st);
        if (s != IDA_OK) return s;
        float *const to[3] = {static_cast<float *>(dw_gate), static_cast<float *>(dw_up), static_cast<float *>(dw_down)};
        float *const sums = reinterpret_cast<float *>(ws + sp.dws);
        const int n = ffn_simt_parts(rows, D, F);
        SimtArgs b = {{fg, fu, fy}, {fx, fx, fa + 2 * tf}, {F, F, D}, {ldx, ldx, F}, {to[0], to[1], to[2]}, nullptr, nullptr,
                      {F, F, D}, {D, D, F}, rows, 3, 1, n, (long long)(3 * df)};
        if (n > 1)
            for (int p = 0; p < 3; ++p) b.out[p] = sums + p * df;
        s = ffn_simt(1, 1, kPlain, b, st);
        if (s == IDA_OK && n > 1) s = ffn_simt_add(sums, to, (long long)df, n, st);
        if (s != IDA_OK) return s;
        SimtArgs c = {{fg, fu}, {static_cast<const float *>(w_gate), static_cast<const float *>(w_up)}, {F, F}, {D, D},
                      {static_cast<float *>(dx)}, nullptr, nullptr, {rows}, {D}, F, 1, 2, 1, 0};
        return ffn_simt(0, 1, kPlain, c, st);
    }
    const int parts = dtype == IDA_BF16 ? 1 : 3;
    Operand X = {x, parts, rows, D, ldx}, Wg = {w_gate, parts, F, D, D}, Wu = {w_up, parts, F, D, D}, Wd = {w_down, parts, D, F, F},
            H = {ac + 2 * tf * es, parts, rows, F, F}, dY = {dout, parts, rows, D, D}, dG = {dg, parts, rows, F, F},
            dU = {du, parts, rows, F, F};
    if (dtype == IDA_F32) {
        SplitArgs a = {{static_cast<const float *>(x), static_cast<const float *>(w_gate), static_cast<const float *>(w_up),
                        static_cast<const float *>(w_down)},
                       {}, {rows, F, F, D}, {ldx, D, D, F}, {D, D, D, F}};
        const size_t at[4] = {sp.xs, sp.wg, sp.wu, sp.wd};
        for (int i = 0; i < 4; ++i) a.dst[i] = reinterpret_cast<__nv_bfloat16 *>(ws + at[i]);
        s = launch_split(a, 4, num_sms, st);
        if (s != IDA_OK) return s;
        X.p = a.dst[0], Wg.p = a.dst[1], Wu.p = a.dst[2], Wd.p = a.dst[3], H.p = ws + sp.hs, dY.p = ws + sp.dys;
        dG.p = ws + sp.dgs, dU.p = ws + sp.dus;
        X.ld = D;
        SplitArgs b = {{reinterpret_cast<const float *>(ac + 2 * tf * es), static_cast<const float *>(dout)},
                       {reinterpret_cast<__nv_bfloat16 *>(ws + sp.hs), reinterpret_cast<__nv_bfloat16 *>(ws + sp.dys)},
                       {rows, rows}, {F, D}, {F, D}};
        s = launch_split(b, 2, num_sms, st);
        if (s != IDA_OK) return s;
    }
    GemmArgs g = {};  // dh, and dg and du of it
    g.problems = 1;
    g.M[0] = rows, g.N[0] = F;
    g.kblocks = (D + 63) / 64;
    add_segments(g, dtype, 0, 0);
    s = operand_map(&g.a[0], dY, 0);
    if (s == IDA_OK) s = operand_map(&g.b[0], Wd, 1);
    if (s == IDA_OK) s = box_map(&g.e[0], ac, dtype, rows, F);
    if (s == IDA_OK) s = box_map(&g.e[1], ac + tf * es, dtype, rows, F);
    if (s == IDA_OK) s = box_map(&g.o[0], dg, dtype, rows, F);
    if (s == IDA_OK) s = box_map(&g.o[1], du, dtype, rows, F);
    if (s == IDA_OK) s = run_gemm(0, 1, kGateBwd, g, dtype, num_sms, st);
    if (s != IDA_OK) return s;
    if (dtype == IDA_F32) {
        SplitArgs a = {{reinterpret_cast<const float *>(dg), reinterpret_cast<const float *>(du)},
                       {reinterpret_cast<__nv_bfloat16 *>(ws + sp.dgs), reinterpret_cast<__nv_bfloat16 *>(ws + sp.dus)},
                       {rows, rows}, {F, F}, {F, F}};
        s = launch_split(a, 2, num_sms, st);
        if (s != IDA_OK) return s;
    }
    GemmArgs w = {};  // the weights' gradients, contracted over rows
    w.problems = 3;
    w.kblocks = (rows + 63) / 64;
    add_segments(w, dtype, 0, 0);
    const Operand *wa[3] = {&dG, &dU, &dY}, *wb[3] = {&X, &X, &H};
    for (int p = 0; p < 3; ++p) {
        w.M[p] = (int)wa[p]->cols, w.N[p] = (int)wb[p]->cols;
        w.out[p] = dw[p];
        if (s == IDA_OK) s = operand_map(&w.a[p], *wa[p], 1);
        if (s == IDA_OK) s = operand_map(&w.b[p], *wb[p], 1);
    }
    if (s == IDA_OK) s = run_gemm(1, 1, kPlain, w, dtype, num_sms, st);
    if (s != IDA_OK) return s;
    GemmArgs d = {};  // dx
    d.problems = d.back = 1;
    d.M[0] = rows, d.N[0] = D;
    d.kblocks = (F + 63) / 64;
    add_segments(d, dtype, 0, 0);
    add_segments(d, dtype, 1, 1);
    s = operand_map(&d.a[0], dG, 0);
    if (s == IDA_OK) s = operand_map(&d.a[1], dU, 0);
    if (s == IDA_OK) s = operand_map(&d.b[0], Wg, 1);
    if (s == IDA_OK) s = operand_map(&d.b[1], Wu, 1);
    d.out[0] = dx;
    if (s == IDA_OK) s = run_gemm(0, 1, kPlain, d, dtype, num_sms, st);
    return s;
}

}  // extern "C"
