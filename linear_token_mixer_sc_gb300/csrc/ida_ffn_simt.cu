// ida_ffn_simt.cu -- the feed-forward block's fp32 products on the CUDA cores: for few rows, where the
// weights' bytes bound them, and for small sizes, where the tensor cores' three parts, tiles of 256 x 256 and
// extra launches cost more than the arithmetic.
//
// A block makes a tile of 32 x 32 with 256 threads: 64 of them hold it, 4 x 4 each, and four such groups
// share each slab of 64 of the contraction (16 each), so that a small product still has many warps.  Slabs come by
// cp.async, three in flight; their sums meet in shared memory, in a fixed order.
#include "ida_gemm.cuh"
#include "ida_ffn_simt.cuh"

namespace ida {

constexpr int FT = 32, FK = 64, FST = 3;                     // tile, slab, slabs in flight
constexpr int FKP = FK + 4, FTP = FT + 4;                    // padded rows: contraction inside, or outside
constexpr int FOP = FT * FKP > FK * FTP ? FT * FKP : FK * FTP;  // floats of an operand's slab
constexpr int FSMEM = FST * 2 * FOP * 4;
static_assert(256 * 17 <= FST * 2 * FOP, "the sums fit where the slabs were");

__device__ __forceinline__ void copy16(float *dst, const float *src, bool live) {  // zeros where it is not live
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// One operand's slab: rows r0 .. of `rows` (K-major) or columns r0 .. (MN-major), contraction k0 ..
template <int MN>
__device__ __forceinline__ void slab(float *s, const float *p, long long ld, int r0, int rows, int k0, int K, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = t + 256 * i;  // 512 pieces of 4 floats
        if (MN) {
            const int k = e >> 3, r = (e & 7) * 4;
            const bool live = k0 + k < K && r0 + r < rows;
            copy16(s + k * FTP + r, p + (live ? (k0 + k) * ld + r0 + r : 0), live);
        } else {
            const int r = e >> 4, k = (e & 15) * 4;
            const bool live = r0 + r < rows && k0 + k < K;
            copy16(s + r * FKP + k, p + (live ? (r0 + r) * ld + k0 + k : 0), live);
        }
    }
}

// The gate's B slab: 16 rows of either factor's weights.
__device__ __forceinline__ void slab_gate(float *s, const float *p0, const float *p1, long long ld, int r0, int rows, int k0, int K, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = t + 256 * i, r = e >> 4, k = (e & 15) * 4;
        const bool live = r0 + (r & 15) < rows && k0 + k < K;
        copy16(s + r * FKP + k, (i ? p1 : p0) + (live ? (r0 + (r & 15)) * ld + k0 + k : 0), live);
    }
}

// Row (column) i of thread t's four: eight apart where the contraction is inside, neighbours otherwise, so
// that a quarter warp's reads of 16 bytes meet no bank twice.
template <int MN>
__device__ __forceinline__ int place(int t, int i) { return MN ? t * 4 + i : t + 8 * i; }

// Four rows' values at contraction k .. k + 3
template <int MN>
__device__ __forceinline__ void fetch(float (&v)[4][4], const float *s, int t, int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4 *>(MN ? s + (k + i) * FTP + t * 4 : s + (t + 8 * i) * FKP + k);
        const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[MN ? e : i][MN ? i : e] = w[e];
    }
}

// PARTS: a block's part of the contraction is that of blockIdx.y
template <int AMN, int BMN, int EPI, bool PARTS>
__global__ void __launch_bounds__(256) ffn_simt_kernel(SimtArgs g) {
    extern __shared__ float4 raw4[];
    float *sm = reinterpret_cast<float *>(raw4);
    constexpr int COLS = EPI == kGate ? FT / 2 : FT;
    int b = blockIdx.x, p = 0;
    while (true) {
        const int n = (g.M[p] + FT - 1) / FT * ((g.N[p] + COLS - 1) / COLS);
        if (b < n || p + 1 >= g.problems) break;
        b -= n;
        ++p;
    }
    const int tm = (g.M[p] + FT - 1) / FT, row0 = b % tm * FT, col0 = b / tm * COLS, M = g.M[p], N = g.N[p];
    const int t = threadIdx.x, group = t >> 6, tx = t & 7, ty = t >> 3 & 7;
    const int per = (g.K + FK - 1) / FK, all = g.halves * per;
    const int first = PARTS ? (int)((long long)all * blockIdx.y / g.parts) : 0;
    const int slabs = PARTS ? (int)((long long)all * (blockIdx.y + 1) / g.parts) - first : all;
    dependent_wait();  // (letting the next launch start early, too, fills the SMs with its waiting blocks: 509 rows' gradients 22 us, then 40)
    auto load = [&](int i) {
        if (i < slabs) {
            const int h = (first + i) / per, k0 = (first + i - h * per) * FK;
            float *A = sm + i % FST * 2 * FOP, *B = A + FOP;
            slab<AMN>(A, g.a[p + h], g.lda[p + h], row0, M, k0, g.K, t);
            if (EPI == kGate)
                slab_gate(B, g.b[0], g.b[1], g.ldb[0], col0, N, k0, g.K, t);
            else
                slab<BMN>(B, g.b[p + h], g.ldb[p + h], col0, N, k0, g.K, t);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float acc[4][4] = {};
    load(0);
    load(1);
    for (int i = 0; i < slabs; ++i) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        load(i + 2);  // over the slab before this one
        const float *A = sm + i % FST * 2 * FOP, *B = A + FOP;
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            float x[4][4], y[4][4];
            fetch<AMN>(x, A, ty, group * 16 + k);
            fetch<BMN>(y, B, tx, group * 16 + k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(x[r][e], y[c][e], acc[r][c]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sm[t * 17 + r * 4 + c] = acc[r][c];
    __syncthreads();
    // thread t now has row `group` of the four of its place
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        v[c] = sm[(t & 63) * 17 + group * 4 + c];
#pragma unroll
        for (int k = 1; k < 4; ++k) v[c] += sm[((t & 63) + 64 * k) * 17 + group * 4 + c];
    }
    const int row = row0 + place<AMN>(ty, group);
    if (row >= M) return;
    if constexpr (EPI == kPlain) {
        float *o = g.out[p] + (PARTS ? blockIdx.y * g.part_floats : 0) + (long long)row * N;
        if (BMN) {
            if (col0 + tx * 4 < N) *reinterpret_cast<float4 *>(o + col0 + tx * 4) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (col0 + tx + 8 * c < N) o[col0 + tx + 8 * c] = v[c];
        }
    } else if constexpr (EPI == kGate) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = col0 + tx + 8 * c;
            if (col >= N) continue;
            const long long at = (long long)row * N + col;
            g.out[0][at] = v[c] * sigmoid<float>(v[c]) * v[c + 2];
            if (g.out[1]) {
                g.out[1][at] = v[c];
                g.out[2][at] = v[c + 2];
            }
        }
    } else {
        const int col = col0 + tx * 4;
        if (col >= N) return;
        const long long at = (long long)row * N + col;
        const float4 x = *reinterpret_cast<const float4 *>(g.gate + at), y = *reinterpret_cast<const float4 *>(g.up + at);
        float dg[4] = {x.x, x.y, x.z, x.w}, du[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) gate_grads<float>(v[c], dg[c], du[c]);
        *reinterpret_cast<float4 *>(g.out[0] + at) = make_float4(dg[0], dg[1], dg[2], dg[3]);
        *reinterpret_cast<float4 *>(g.out[1] + at) = make_float4(du[0], du[1], du[2], du[3]);
    }
}

template <int AMN, int BMN, int EPI, bool PARTS = false>
static ida_status launch_simt(const SimtArgs &a, cudaStream_t st) {
    constexpr int cols = EPI == kGate ? FT / 2 : FT;
    long long blocks = 0;
    for (int p = 0; p < a.problems; ++p) blocks += (long long)((a.M[p] + FT - 1) / FT) * ((a.N[p] + cols - 1) / cols);
    const auto kernel = ffn_simt_kernel<AMN, BMN, EPI, PARTS>;
    cudaError_t e = allow_smem(kernel, FSMEM);
    if (e == cudaSuccess) e = launch_dependent(kernel, dim3((unsigned)blocks, PARTS ? (unsigned)a.parts : 1), dim3(256), FSMEM, st, a);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("fp32 product launch: ") + cudaGetErrorString(e));
    return launched("fp32 product");
}

ida_status ffn_simt(int a_mn, int b_mn, int epi, const SimtArgs &a, cudaStream_t st) {
    if (epi == kGate) return launch_simt<0, 0, kGate>(a, st);
    if (epi == kGateBwd) return launch_simt<0, 1, kGateBwd>(a, st);
    if (a_mn) return a.parts > 1 ? launch_simt<1, 1, kPlain, true>(a, st) : launch_simt<1, 1, kPlain>(a, st);
    if (b_mn) return launch_simt<0, 1, kPlain>(a, st);
    return launch_simt<0, 0, kPlain>(a, st);
}

// One block's slabs run one behind the other, some 0.7 us each, so few tiles over many rows are shared by as many blocks
// as the SMs hold at once (four each), of at least eight slabs; their sums are added in a launch of its own, in order.
// (Gradients of 2^21 rows of 8 and 8 channels 24353 us in whole, now 1391; of 16384 of 32 and 64 204 and 31, 2048 of them 32
// and 15.)  A sum in one thread then has fewer terms, too.
int ffn_simt_parts(long long T, long long D, long long F) {
    const long long tiles = 3 * ((D + FT - 1) / FT) * ((F + FT - 1) / FT), slabs = (T + FK - 1) / FK;
    const long long n = 608 / tiles < slabs / 8 ? 608 / tiles : slabs / 8;
    return n > 1 ? (int)n : 1;
}

__global__ void __launch_bounds__(128) simt_add_kernel(const float4 *from, float4 *o0, float4 *o1, float4 *o2, long long n, int parts) {
    const long long e = (long long)blockIdx.x * 128 + threadIdx.x;  // n: pieces of 4 floats in an output
    dependent_wait();
    if (e >= 3 * n) return;
    float4 s = from[e];
    for (int k = 1; k < parts; ++k) {
        const float4 v = from[k * 3 * n + e];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    (e < n ? o0 : e < 2 * n ? o1 : o2)[e % n] = s;
}

ida_status ffn_simt_add(const float *from, float *const (&out)[3], long long n, int parts, cudaStream_t st) {
    const long long blocks = (3 * n / 4 + 127) / 128;
    const cudaError_t e = launch_dependent(simt_add_kernel, dim3((unsigned)blocks), dim3(128), 0, st, reinterpret_cast<const float4 *>(from),
                                           reinterpret_cast<float4 *>(out[0]), reinterpret_cast<float4 *>(out[1]),
                                           reinterpret_cast<float4 *>(out[2]), n / 4, parts);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("fp32 sums launch: ") + cudaGetErrorString(e));
    return launched("fp32 sums");
}

}  // namespace ida
