// ida_skinny.cu -- the feed-forward block's and the 8-bit products for a few rows (decoding), where
// the weights' bytes bound them.
//
// Every weight is read once, 16 bytes a lane straight into the registers of a matrix instruction: the
// weights are its 16 x K operand, the rows (tokens) its 8 columns, so the tile that tcgen05 would want
// (128 weights' rows at least, through shared memory) is not needed and the loads of all warps of all SMs
// are in flight at once.  A quad of lanes reads 64 bytes of a weight's row; the instruction's order of the
// contraction is any one order that both operands share, so a lane's 16 bytes serve two instructions.
// The warps of a block share its weights' rows and split the contraction; their sums meet in shared
// memory, in a fixed order.  The gate's kernel pairs 8 rows of each weight in one instruction, so that both factors of a
// product come out in the same block.  Few weights' rows are spread over more blocks, 8 to a block.
#include "ida_gemm.cuh"
#include "ida_skinny.cuh"

namespace ida {

__device__ __forceinline__ void mma_rows(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         bool e4m3) {
    if (e4m3)
        asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the value at the same place of the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ float remote_float(const float *p, int rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Warps of a block and, below, chunks of 128 bytes that a lane has in flight: in bf16 16 warps of two tiles' rows (one
// row through the block of 2048 and 5632 channels 2.6 us less than by 8, of 17.5 now), in e4m3 8.
constexpr int skinny_warps(bool e8) { return e8 ? 8 : 16; }

// SUB tiles of 16 weights' rows a block, of which a plain product may use 8 (HALVES
// 1).  GATE: rows 8 .. 15 of a tile are w1's.  E8 && GATE: a cluster of 8 blocks makes the 128 channels of
// a scale.
// The gate's product in bf16 leaves its block in two bf16 parts, 16 bits in all, and the product back takes both
// (WIDE), for two instructions each on weights that are there anyway: of few rows one rounding of the product
// would be seen in the result (one row's error 2.3e-3 of its size, now 1.6e-3, which is the output's rounding;
// 0.6 us of 17.5 with 2048 and 5632 channels, 0.9 of 18.9 for eight rows).
template <bool E8, int SUB, int HALVES, bool GATE, bool WIDE>
__global__ void __launch_bounds__(skinny_warps(E8) * 32, E8 ? 1 : 2) skinny_kernel(SkinnyArgs a) {
    constexpr int U = SUB * HALVES >= 2 ? 1 : 2, LD = 9, ES = E8 ? 1 : 2;
    constexpr int COLS = SUB * (GATE ? 8 : 8 * HALVES);  // output columns of a block
    extern __shared__ float red[];  // [warps][SUB][16][LD]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, nw = blockDim.x >> 5;
    const long long n0 = (long long)blockIdx.x * COLS;
    const long long kbytes = (long long)a.K * ES;
    const int chunks = (int)((kbytes + 127) / 128);
    const char *row[SUB][HALVES];
#pragma unroll
    for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            long long r = n0 + (GATE ? 8 * s : 8 * HALVES * s + 8 * h) + g;
            if (r >= a.N) r = a.N - 1;  // not stored
            row[s][h] = static_cast<const char *>(GATE && h ? a.w1 : a.w0) + r * kbytes;
        }
    float acc[SUB][4];
#pragma unroll
    for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[s][i] = 0.f;

    uint4 w[U][SUB][HALVES][2];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * nw;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const long long at = (long long)c * 128 + j * 64 + t * 16;
#pragma unroll
                for (int s = 0; s < SUB; ++s)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        w[u][s][h][j] = c < chunks && at < kbytes ? __ldcs(reinterpret_cast<const uint4 *>(row[s][h] + at)) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    // The launch before may make any of these inputs (none of their loads is one of read-only data, which might be
    // moved up before the wait).  A product that follows the gate's in one call reads its first weights while that one
    // adds up its sums: it let this one start only after it had waited for all before it.
    if (!a.weights_ready) dependent_wait();
    fetch(warp);
    if (a.weights_ready) dependent_wait();
    for (int c0 = warp; c0 < chunks; c0 += U * nw) {
        if (c0 != warp) fetch(c0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * nw;
            if (c >= chunks) break;
            uint4 x[2], rest[2];  // rest: x's second parts (WIDE)
            float m[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const long long at = (long long)c * 128 + j * 64 + t * 16;
                const bool in = g < a.T && at < kbytes;
                const char *src = static_cast<const char *>(a.x) + g * a.ldx * ES + at;
                x[j] = in ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                if (WIDE) rest[j] = in ? *reinterpret_cast<const uint4 *>(src + a.T * a.ldx * ES) : make_uint4(0, 0, 0, 0);
                if (E8) m[j] = 2 * t + j < a.T ? a.sa[(long long)(2 * t + j) * chunks + c] : 0.f;
            }
            float s0 = 1.f, s1 = 1.f;
            if (E8) {
                const long long blk = n0 / 128 * chunks + c;
                s0 = a.s0[blk];
                s1 = GATE ? a.s1[blk] : s0;
            }
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                float(&d)[4] = E8 ? part : acc[s];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 lo = w[u][s][0][j], hi = HALVES == 2 ? w[u][s][HALVES - 1][j] : make_uint4(0, 0, 0, 0);
                    mma_rows(d, lo.x, hi.x, lo.y, hi.y, x[j].x, x[j].y, E8);
                    mma_rows(d, lo.z, hi.z, lo.w, hi.w, x[j].z, x[j].w, E8);
                    if (WIDE) {
                        mma_rows(d, lo.x, hi.x, lo.y, hi.y, rest[j].x, rest[j].y, E8);
                        mma_rows(d, lo.z, hi.z, lo.w, hi.w, rest[j].z, rest[j].w, E8);
                    }
                }
                if (E8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[s][i] = fmaf(part[i], m[i & 1] * (i < 2 ? s0 : s1), acc[s][i]);
            }
        }
    }
    // The product back may read its weights from here on.  (One row through the block of 2048 and 5632 channels 18.0 us,
    // now 17.5, and the gate in 8 bits 10.3 and 10.0; a product's own early end, let in for the next call's gate, which
    // only waits, cost 0.3 us of 768 and 2048 channels' 4.6, and one ahead of the loop won nothing.)
    if (GATE) dependent_launch();
#pragma unroll
    for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((warp * SUB + s) * 16 + g + (i >> 1) * 8) * LD + 2 * t + (i & 1)] = acc[s][i];
    __syncthreads();
    auto sum = [&](int s, int r, int tok) {
        float v = red[(s * 16 + r) * LD + tok];
        for (int k = 1; k < nw; ++k) v += red[((k * SUB + s) * 16 + r) * LD + tok];
        return v;
    };
    if constexpr (!GATE) {
        for (int i = threadIdx.x; i < COLS * a.T; i += blockDim.x) {
            const int tok = i / COLS, c = i % COLS;
            if (n0 + c >= a.N) continue;
            const float v = sum(c / (8 * HALVES), c % (8 * HALVES), tok);
            const long long at = tok * a.N + n0 + c;
            if (a.out_f32)
                static_cast<float *>(a.out)[at] = v;
            else
                static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
        }
    } else if constexpr (!E8) {
        for (int i = threadIdx.x; i < COLS * a.T; i += blockDim.x) {
            const int tok = i / COLS, c = i % COLS;
            const float x = sum(c / 8, c % 8, tok), y = sum(c / 8, 8 + c % 8, tok);
            const long long at = tok * a.N + n0 + c;
            const float h = x * sigmoid<__nv_bfloat16>(x) * y;
            const long long part = (long long)a.T * a.N;
            // (the first part towards zero where the nearest is not finite)
            const __nv_bfloat16 hi = __float2bfloat16_rn(h), first = fabsf(h) < 0x1.FFp127f ? hi : __float2bfloat16_rz(h);
            static_cast<__nv_bfloat16 *>(a.out)[at] = first;
            static_cast<__nv_bfloat16 *>(a.out)[at + part] = __float2bfloat16_rn(h - __bfloat162float(first));
            if (a.acts) {
                static_cast<__nv_bfloat16 *>(a.acts)[at] = __float2bfloat16_rn(x);
                static_cast<__nv_bfloat16 *>(a.acts)[at + part] = __float2bfloat16_rn(y);
                static_cast<__nv_bfloat16 *>(a.acts)[at + 2 * part] = hi;
            }
        }
    } else {
        // 16 channels of a row are 16 lanes'; the 8 blocks of a cluster have the 128 of a scale
        __shared__ float top[8];
        const int c = threadIdx.x & 15, tok = threadIdx.x >> 4;
        float v = 0.f;
        if (tok < a.T && n0 + c < a.N) {
            const float x = sum(c / 8, c % 8, tok), y = sum(c / 8, 8 + c % 8, tok);
            v = x * sigmoid<__nv_bfloat16>(x) * y;
        }
        float m = fabsf(v);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (c == 0 && tok < 8) top[tok] = m;
        cluster_sync_all();
        if (tok < a.T) {
            for (int r = 0; r < 8; ++r) m = fmaxf(m, remote_float(&top[tok], r));
            const float sc = quant_scale(m);
            if (n0 + c < a.N)
                static_cast<uint8_t *>(a.out)[tok * (long long)a.N + n0 + c] = Quotient(sc).one(v);
            if (cluster_rank() == 0 && c == 0) a.so[(long long)tok * ((a.N + 127) / 128) + n0 / 128] = sc;
        }
        cluster_sync_all();  // the maxima have been read
    }
}

template <bool E8, int SUB, int HALVES, bool GATE, bool WIDE = !E8 && !GATE>
static ida_status launch_skinny(const SkinnyArgs &a, cudaStream_t st) {
    constexpr int cols = SUB * (GATE ? 8 : 8 * HALVES);
    const auto kernel = skinny_kernel<E8, SUB, HALVES, GATE, WIDE>;
    const long long chunks = ((long long)a.K * (E8 ? 1 : 2) + 127) / 128;
    // the 8-bit gate's threads make 16 channels of up to 8 rows
    constexpr int most = skinny_warps(E8);
    const int warps = E8 && GATE ? most : chunks < most ? (int)chunks : most;
    const size_t smem = (size_t)warps * SUB * 16 * 9 * sizeof(float);
    cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    const unsigned blocks = (unsigned)((a.N + cols - 1) / cols);
    cfg.gridDim = dim3(E8 && GATE ? (blocks + 7) / 8 * 8 : blocks);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 8;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = E8 && GATE ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("few rows' product launch: ") + cudaGetErrorString(e));
    return launched("few rows' product");
}

// fp32 on the CUDA cores: a block's warps share four rows of weights (two of either factor) and split the
// contraction, a lane taking four of each 128; every lane has sums for all rows of x.
template <int NT, bool GATE>
__global__ void __launch_bounds__(256) skinny_f32_kernel(SkinnyArgs a) {
    constexpr int U = 2;
    __shared__ float red[8][4 * NT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n0 = (long long)blockIdx.x * (GATE ? 2 : 4);
    const float *row[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        row[r] = static_cast<const float *>(GATE && r >= 2 ? a.w1 : a.w0) + (n0 + (GATE ? r & 1 : r)) * a.K + lane * 4;
    const float *x = static_cast<const float *>(a.x) + lane * 4;
    float acc[4][NT] = {};
    float4 w[U][4];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int k = k0 + u * 1024;
                w[u][r] = k + lane * 4 < a.K ? __ldcs(reinterpret_cast<const float4 *>(row[r] + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
    };
    if (!a.weights_ready) dependent_wait();
    fetch(warp * 128);
    if (a.weights_ready) dependent_wait();
    for (int k0 = warp * 128; k0 < a.K; k0 += U * 1024) {
        if (k0 != warp * 128) fetch(k0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * 1024;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t < a.T && k + lane * 4 < a.K) v = *reinterpret_cast<const float4 *>(x + t * a.ldx + k);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[r][t] = fmaf(w[u][r].w, v.w, fmaf(w[u][r].z, v.z, fmaf(w[u][r].y, v.y, fmaf(w[u][r].x, v.x, acc[r][t]))));
            }
        }
    }
    dependent_launch();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float v = warp_sum(acc[r][t]);
            if (lane == 0) red[warp][r * NT + t] = v;
        }
    __syncthreads();
    auto sum = [&](int i) {
        float v = red[0][i];
        for (int k = 1; k < 8; ++k) v += red[k][i];
        return v;
    };
    constexpr int COLS = GATE ? 2 : 4;
    const int t = threadIdx.x / COLS, c = threadIdx.x % COLS;
    if (t >= a.T) return;
    const long long at = t * (long long)a.N + n0 + c;
    if (GATE) {
        const float g = sum(c * NT + t), u = sum((2 + c) * NT + t);
        const float h = g * sigmoid<float>(g) * u;
        static_cast<float *>(a.out)[at] = h;
        if (a.acts) {
            const long long part = (long long)a.T * a.N;
            static_cast<float *>(a.acts)[at] = g;
            static_cast<float *>(a.acts)[at + part] = u;
            static_cast<float *>(a.acts)[at + 2 * part] = h;
        }
    } else {
        static_cast<float *>(a.out)[at] = sum(c * NT + t);
    }
}

template <int NT, bool GATE>
static ida_status launch_f32(const SkinnyArgs &a, cudaStream_t st) {
    const cudaError_t e = launch_dependent(skinny_f32_kernel<NT, GATE>, dim3((unsigned)(a.N / (GATE ? 2 : 4))), dim3(256), 0, st, a);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("few rows' product launch: ") + cudaGetErrorString(e));
    return launched("few rows' product");
}
template <bool GATE>
static ida_status launch_f32_rows(const SkinnyArgs &a, cudaStream_t st) {
    return a.T <= 2 ? launch_f32<2, GATE>(a, st) : launch_f32<8, GATE>(a, st);
}

ida_status skinny_product(const SkinnyArgs &a, int type, int num_sms, cudaStream_t st) {
    if (type == kFewF32) return launch_f32_rows<false>(a, st);
    // 16 rows of weights to a block where that leaves every SM two of them
    if (a.N >= 32 * num_sms) return type == kFewE4M3 ? launch_skinny<true, 1, 2, false>(a, st) : launch_skinny<false, 1, 2, false>(a, st);
    return type == kFewE4M3 ? launch_skinny<true, 1, 1, false>(a, st) : launch_skinny<false, 1, 1, false>(a, st);
}
ida_status skinny_gate(const SkinnyArgs &a, int type, cudaStream_t st) {
    if (type == kFewF32) return launch_f32_rows<true>(a, st);
    return type == kFewE4M3 ? launch_skinny<true, 2, 2, true>(a, st) : launch_skinny<false, 1, 2, true>(a, st);
}

}  // namespace ida
