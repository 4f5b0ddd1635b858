// ida_ssm_chunk.cu -- the selective scan in chunks on the tcgen05 tensor cores (bf16 inputs).
//
// Over a chunk of Q = 128 positions, with S_t the sum of log2 a up to position t of it, X_0 the
// state before it and X_Q the state behind it (see ida_ssm.cuh for the recurrence):
//   G    [t][s]  = c_t . b_s                                   MMA, K = M
//   P    [t][s]  = G 2^(S_t - S_s) D_s (s <= t), + D at s = t  CUDA cores, G from TMEM, P to TMEM
//   Y    [t][j]  = P x + (c_t 2^S_t) X_0                       MMA, K = Q and K = M
//   X_Q^T [j][m] = 2^S_Q X_0^T + x^T (b_s 2^(S_Q - S_s) D_s)   scaled in TMEM, then MMA, K = Q
// No factor exceeds 1 (but D_s): decays are differences of S taken before the exponential.
//
// Precision.  Everything accumulates in fp32.  P, c 2^S and the X_0 operand are rounded to bf16
// (2^-9 of a term on average, below y's own rounding); the scaled b of the state update is kept as
// the sum of two bf16 tiles, because the state is an fp32 result that the next segment, call or
// decode step continues.  S is summed in 2^-32 fixed point: it is exact over any chunk or segment.
//
// One CTA of 256 threads walks the chunks of one (row, head, up to 128 channels, segment).  x, b
// and c tiles arrive by TMA with the 128-byte swizzle that the MMA descriptors name, so one copy
// serves as a K-major operand (b, c in G) and as an MN-major one (x, b in the state update, whose K
// is the position).  P is an A operand in TMEM: thread t of a lane quarter makes row t of it from
// row t of G.  The state stays in TMEM; y leaves through shared memory that is dead by then, by TMA.
// With M <= 64 two CTAs share an SM (256 TMEM columns and 101 KB each) and fill each other's
// waits: a chunk is a chain of copy, MMA, CUDA-core stage, MMA, epilogue.
//
// Few (row, head) units do not fill the SMs: sequences are cut into segments, whose last states
// from zero a first launch leaves in the workspace (x and b only, the state update alone); each
// segment then starts from the decayed sum of those before it.
//
// Every wait is bounded.  On a timeout all threads of the CTA leave the loop together, the kernel
// records kErrWaitTimeout, waits (bounded) for its copy in flight, frees its TMEM and returns.
#include <cuda.h>

#include <mutex>

#include "ida_ssm.cuh"
#include "tc_sm103.cuh"

namespace ida {

using namespace tc;

constexpr int SQ = 128;         // positions per chunk
constexpr int SSLAB = SQ * 128; // bytes of 128 rows of 64 bf16
constexpr int STH = 256;        // threads per CTA

// Shared memory map; DP, MP: channels and state rows rounded up to 64 or 128.
template <int DP, int MP, bool STATE>
struct SsmSmem {
    static constexpr int X = 0;                            // [DP / 64][128 s][64] bf16
    static constexpr int B = X + DP / 64 * SSLAB;          // [MP / 64][128 s][64]: b, then its scaled high part
    static constexpr int LO = B + MP / 64 * SSLAB;         // the scaled low part
    static constexpr int C = LO + MP / 64 * SSLAB;         // [MP / 64][128 t][64]: c, then scaled
    static constexpr int SBS = DP * 128;                   // bytes of one slab of SB
    static constexpr int SB = C + (STATE ? 0 : MP / 64 * SSLAB);  // [MP / 64][DP j][64]: X_0^T
    static constexpr int MISC = SB + (STATE ? 0 : MP / 64 * SBS);
    // the output tile [DP / 64][128 t][64] goes over SB and LO, which no copy writes to
    static constexpr int OUT0 = MP / 64 * SBS >= SSLAB ? SB : LO;
    static constexpr int OUT1 = MP == 128 ? SB + SSLAB : LO;
    static constexpr int ARR = MISC + 64;                  // 5 arrays of 128 floats, 8 floats
    static constexpr int TOT = ARR + 5 * SQ * 4 + 8 * 4;   // 4 64-bit totals
    static constexpr int TOTAL = TOT + 32;
};

template <int DP, int MP>
struct SsmTmem {
    static constexpr uint32_t G = 0;    // [t][s], later Y [t][j]
    static constexpr uint32_t P = 128;  // [t][s] bf16 pairs
    static constexpr uint32_t S = 192;  // [j][m]; with DP = 64 lanes 64.. repeat 0..63
    static constexpr uint32_t COLS = MP == 64 ? 256 : 512;
};

// Shared-memory descriptor of a 128-byte-swizzled operand whose 64-element rows are 128 bytes
// apart: `sbo` 1024 between groups of 8 rows; `lbo` between 64-element slabs (MN-major operands).
__device__ __forceinline__ SmemDesc sw_desc(uint32_t addr, uint32_t lbo) {
    return {((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16), (1024u >> 4) | (1u << 14) | (2u << 29)};
}
__device__ __forceinline__ SmemDesc sw_step(SmemDesc d, uint32_t bytes) {
    d.lo += bytes >> 4;
    return d;
}
// byte offset of 16-byte piece `c` of row `r` in such a slab
__device__ __forceinline__ int sw_off(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void mma_f16_t(uint32_t d, uint32_t a_tmem, SmemDesc b, uint32_t id, uint32_t acc) {
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

constexpr float kFix = 4294967296.f, kUnfix = 1.f / 4294967296.f;  // 2^32

template <int DP, int MP, bool STATE>
__global__ void __launch_bounds__(STH, STATE ? 3 : (MP == 64 ? 2 : 1))
    ssm_chunk_kernel(ScanArgs a, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y) {
    using L = SsmSmem<DP, MP, STATE>;
    using T = SsmTmem<DP, MP>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);  // 0 copies, 1 G, 2 Y and state
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 48);
    float *cumf = reinterpret_cast<float *>(sm + L::ARR);  // S_t
    float *uf = cumf + SQ;                                 // S_s - log2 D_s
    float *rs = uf + SQ;                                   // 2^(S at the end of s's block of 16 - uf)
    float *wst = rs + SQ;                                  // 2^(S_Q - S_s) D_s
    float *et = wst + SQ;                                  // 2^S_t
    float *cref = et + SQ;                                 // S at the end of each block of 16
    long long *tot = reinterpret_cast<long long *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q4 = warp & 3, half = warp >> 2, tl = 32 * q4 + lane;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d;
    const int slices = (d + DP - 1) / DP, nseg = STATE ? a.segs - 1 : a.segs;
    int id = blockIdx.x;
    const int seg = id % nseg;
    id /= nseg;
    const int j0 = id % slices * DP, unit = id / slices, b = unit / H, h = unit % H, g = h / (H / a.G);
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg), nch = (t_end - t_begin + SQ - 1) / SQ;
    const __nv_bfloat16 *gdt = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)b * N * a.lddt + h;
    const float rate2 = expf(a.a_log[h]) * 1.4426950408889634f, dt_bias = a.dt_bias[h];
    const float skip = STATE ? 0.f : a.D[h];
    constexpr uint32_t TILE_BYTES = (uint32_t)SSLAB * (DP / 64 + MP / 64 * (STATE ? 1 : 2));
    constexpr uint32_t S_COL = STATE ? 0 : T::S, COLS = STATE ? MP : T::COLS;

    if ((s0 & 1023u) != 0u) {  // the swizzle repeats every 1024 bytes
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_b);
        if (!STATE) {
            tma_prefetch_desc(&tm_c);
            tma_prefetch_desc(&tm_y);
        }
    }
    if (warp == 0) {
        tmem_alloc(tslot, COLS);
        tmem_relinquish();
    }
    const auto fetch = [&](int t0) {  // thread 0
        mbar_arrive_expect_tx(&bar[0], TILE_BYTES);
#pragma unroll
        for (int i = 0; i < MP / 64; ++i) {
            tma_load_4d(sm + L::B + i * SSLAB, &tm_b, 64 * i, g, t0, b, &bar[0]);
            if (!STATE) tma_load_4d(sm + L::C + i * SSLAB, &tm_c, 64 * i, g, t0, b, &bar[0]);
        }
#pragma unroll
        for (int i = 0; i < DP / 64; ++i) tma_load_4d(sm + L::X + i * SSLAB, &tm_x, j0 + 64 * i, h, t0, b, &bar[0]);
    };
    float dt_next = 0.f;  // threads 0..127: the raw step of my position of the coming chunk
    const auto fetch_dt = [&](int t0) {
        if (tid < SQ) dt_next = t0 + tid < t_end ? __bfloat162float(gdt[(size_t)(t0 + tid) * a.lddt]) : 0.f;
    };
    fetch_dt(t_begin);
    __syncthreads();
    if (tid == 0) fetch(t_begin);
    tc_fence_after();
    const uint32_t tm = *tslot;
    const int ch = DP == 64 ? (tl & 63) : tl;  // my channel of the state tile
    constexpr int MH = MP / 2;                 // state rows of a warp half
    {
        // the state before the segment: the given one and the segments before, decayed
        const bool mine = j0 + ch < d;
        float v[16];
#pragma unroll
        for (int blk = 0; blk < MH / 16; ++blk) {
            const int m0 = half * MH + 16 * blk;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
            if (!STATE)
                for (int s = -1; s < seg; ++s) {
                    const float *p = s >= 0 ? a.seg_state + ((size_t)unit * a.segs + s) * M * d
                                            : (a.state_in ? a.state_in + (size_t)unit * M * d : nullptr);
                    if (!p || !mine) continue;
                    const float f = s < 0 ? 0.f : ex2(a.seg_log[(size_t)unit * a.segs + s]);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (m0 + e < M) v[e] = fmaf(f, v[e], __ldg(p + (size_t)(m0 + e) * d + j0 + ch));
                }
            tmem_st16(tm + lane_base + S_COL + m0, v);
        }
        tmem_wait_st();
    }
    long long seg_total = 0;
    bool ok = true;
    int i = 0;
    for (; i < nch; ++i) {
        const int t0 = t_begin + i * SQ;
        const uint32_t par = i & 1;
        // running sum of log2 a: each warp's, then all
        float delta = 0.f;
        long long fx = 0, own = 0;
        if (tid < SQ) {
            if (t0 + tid < t_end) delta = softplus(dt_next + dt_bias);  // behind the end nothing decays or is added
            own = fx = __float2ll_rn(fmaxf(-rate2 * delta, -1048576.f) * kFix);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, fx, o);
                if (lane >= o) fx += u;
            }
            if (lane == 31) tot[warp] = fx;
        }
        if (!STATE && tid == 0) bulk_wait_read_all();  // y of the last chunk has left SB and LO
        ok = mbar_wait(&bar[0], par);
        if (__syncthreads_or(!ok)) break;
        if (!STATE && tid == 0) {
            tc_fence_after();
            const SmemDesc da = sw_desc(s0 + L::C, 16), db = sw_desc(s0 + L::B, 16);
            constexpr uint32_t id_g = idesc(128, 128, 1, 1);
#pragma unroll
            for (int k = 0; k < MP / 16; ++k) {
                const uint32_t off = (k / 4) * SSLAB + (k % 4) * 32;
                mma_f16(tm + T::G, sw_step(da, off), sw_step(db, off), id_g, k > 0);
            }
            mma_commit(&bar[1]);
        }
        const long long t1 = tot[0], t2 = t1 + tot[1], t3 = t2 + tot[2], all = t3 + tot[3];
        const float decay = ex2((float)all * kUnfix);
        seg_total += all;
        if (tid < SQ) {
            fx += warp == 0 ? 0 : warp == 1 ? t1 : warp == 2 ? t2 : t3;
            const float s = (float)fx * kUnfix;
            wst[tid] = ex2((float)(all - fx) * kUnfix) * delta;
            if (!STATE) {
                const float u = s - log2f(delta);  // D = 0: +inf, and 2^(.. - u) = 0
                const float ref = __shfl_sync(0xffffffffu, s, lane | 15);
                cumf[tid] = s;
                uf[tid] = u;
                rs[tid] = ex2(ref - u);
                et[tid] = ex2(s);
                if ((lane & 15) == 15) cref[tid >> 4] = s;
            }
        }
        (void)own;
        // the state: its bf16 copy for Y, then its decay over the chunk
        tc_fence_after();
#pragma unroll
        for (int blk = 0; blk < MH / 16; ++blk) {
            const int m0 = half * MH + 16 * blk;
            float v[16];
            tmem_ld16(tm + lane_base + S_COL + m0, v);
            tmem_wait_ld();
            if (!STATE && tl < DP) {
                unsigned char *row = sm + L::SB + m0 / 64 * L::SBS;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<uint4 *>(row + sw_off(tl, m0 % 64 / 8 + c)) =
                        make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                                   pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= decay;
            tmem_st16(tm + lane_base + S_COL + m0, v);
        }
        if (!STATE) ok = mbar_wait(&bar[1], par);
        if (__syncthreads_or(!ok)) break;  // G is there, and the arrays above
        tc_fence_after();
        if (!STATE) {
            // P: row tl; the two warps of a lane quarter take blocks of 16 columns in turn
            const float ct = cumf[tl];
            for (int kb = half; kb < 8; kb += 2) {
                uint32_t w[8];
                if (kb > 2 * q4 + 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                } else {
                    float v[16];
                    tmem_ld16(tm + lane_base + T::G + 16 * kb, v);
                    tmem_wait_ld();
                    if (kb < 2 * q4) {  // wholly before my rows: one exponential for the block
                        const float f = ex2(ct - cref[kb]);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 r = *reinterpret_cast<const float4 *>(rs + 16 * kb + e);
                            v[e] *= f * r.x;
                            v[e + 1] *= f * r.y;
                            v[e + 2] *= f * r.z;
                            v[e + 3] *= f * r.w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int s = 16 * kb + e;
                            const float p = v[e] * ex2(ct - uf[s]);
                            v[e] = s < tl ? p : s == tl ? p + skip : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                }
                tmem_st8(tm + lane_base + T::P + 8 * kb, w);
            }
        }
        // b 2^(S_Q - S_s) D_s in two parts, c 2^S_t: row r, half of the columns
        {
            const int r = tid & 127, p0 = (tid >> 7) * (MP / 16);
            const float w = wst[r], e = STATE ? 0.f : et[r];
#pragma unroll
            for (int k = 0; k < MP / 16; ++k) {
                const int p = p0 + k, off = p / 8 * SSLAB + sw_off(r, p % 8);
                uint4 *pb = reinterpret_cast<uint4 *>(sm + L::B + off);
                float v[8], hi[8];
                Vec16<__nv_bfloat16>::unpack(*pb, v);
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] *= w;
                const uint4 uh = Vec16<__nv_bfloat16>::pack(v);
                Vec16<__nv_bfloat16>::unpack(uh, hi);
                *pb = uh;
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] -= hi[x];
                *reinterpret_cast<uint4 *>(sm + L::LO + off) = Vec16<__nv_bfloat16>::pack(v);
                if (!STATE) {
                    uint4 *pc = reinterpret_cast<uint4 *>(sm + L::C + off);
                    Vec16<__nv_bfloat16>::unpack(*pc, v);
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] *= e;
                    *pc = Vec16<__nv_bfloat16>::pack(v);
                }
            }
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            const SmemDesc dx = sw_desc(s0 + L::X, SSLAB);  // [K = s][j]
            if (!STATE) {
                constexpr uint32_t id_p = idesc(128, DP, 1, 1, 0, 1), id_s = idesc(128, DP, 1, 1);
#pragma unroll
                for (int k = 0; k < SQ / 16; ++k)
                    mma_f16_t(tm + T::G, tm + T::P + 8 * k, sw_step(dx, k * 2048), id_p, k > 0);
                const SmemDesc dc = sw_desc(s0 + L::C, 16), ds = sw_desc(s0 + L::SB, 16);
#pragma unroll
                for (int k = 0; k < MP / 16; ++k)
                    mma_f16(tm + T::G, sw_step(dc, k / 4 * SSLAB + k % 4 * 32), sw_step(ds, k / 4 * L::SBS + k % 4 * 32),
                            id_s, 1);
            }
            // x^T as A: with DP = 64 its second 64 rows repeat the first
            const SmemDesc da = sw_desc(s0 + L::X, DP == 64 ? 0 : SSLAB);
            const SmemDesc dh = sw_desc(s0 + L::B, SSLAB), dl = sw_desc(s0 + L::LO, SSLAB);
            constexpr uint32_t id_x = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll
            for (int k = 0; k < SQ / 16; ++k) mma_f16(tm + S_COL, sw_step(da, k * 2048), sw_step(dh, k * 2048), id_x, 1);
#pragma unroll
            for (int k = 0; k < SQ / 16; ++k) mma_f16(tm + S_COL, sw_step(da, k * 2048), sw_step(dl, k * 2048), id_x, 1);
            mma_commit(&bar[2]);
        }
        fetch_dt(t0 + SQ);
        ok = mbar_wait(&bar[2], par);
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (tid == 0 && i + 1 < nch) fetch(t0 + SQ);
        if (!STATE) {
            // y: row tl, half of the channels
            constexpr int CW = DP / 2;  // channels of a warp
            unsigned char *out = sm + (DP == 128 && half ? L::OUT1 : L::OUT0);
            const int p0 = DP == 128 ? 0 : half * 4;
#pragma unroll
            for (int blk = 0; blk < CW / 16; ++blk) {
                float v[16];
                tmem_ld16(tm + lane_base + T::G + half * CW + 16 * blk, v);
                tmem_wait_ld();
                *reinterpret_cast<uint4 *>(out + sw_off(tl, p0 + 2 * blk)) = Vec16<__nv_bfloat16>::pack(v);
                *reinterpret_cast<uint4 *>(out + sw_off(tl, p0 + 2 * blk + 1)) = Vec16<__nv_bfloat16>::pack(v + 8);
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
#pragma unroll
                for (int s = 0; s < DP / 64; ++s)
                    if (j0 + 64 * s < d) tma_store_4d(&tm_y, j0 + 64 * s, h, t0, b, sm + (s ? L::OUT1 : L::OUT0));
                bulk_commit();
            }
        }
    }
    if (i < nch) {  // a wait ran out
        if (tid == 0) {
            report_error(a.err, kErrWaitTimeout);
            mbar_wait(&bar[0], i & 1);  // the copy of this chunk, if it is still in flight
        }
    } else {
        float *out = STATE ? a.seg_state + ((size_t)unit * a.segs + seg) * M * d
                           : (a.final_state && seg == a.segs - 1 ? a.final_state + (size_t)unit * M * d : nullptr);
        if (out && (DP == 128 || tl < DP)) {
#pragma unroll
            for (int blk = 0; blk < MH / 16; ++blk) {
                const int m0 = half * MH + 16 * blk;
                float v[16];
                tmem_ld16(tm + lane_base + S_COL + m0, v);
                tmem_wait_ld();
                if (j0 + tl < d)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (m0 + e < M) out[(size_t)(m0 + e) * d + j0 + tl] = v[e];
            }
        }
        if (STATE && tid == 0 && j0 == 0) a.seg_log[(size_t)unit * a.segs + seg] = (float)seg_total * kUnfix;
    }
    if (!STATE && tid == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, COLS);
    }
}

// ---- host side ---------------------------------------------------------------------------

typedef CUresult (*SsmEncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static SsmEncodeFn ssm_encode_fn() {
    static std::once_flag once;
    static SsmEncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<SsmEncodeFn>(p);
    });
    return fn;
}

// Rows of B x N positions, ld elements apart, of K units of w channels each, as a map
// (channel, unit, position, row) with boxes of 64 channels of one unit over 128 positions.  Channels
// behind w and positions behind N are read as zero and not written.
static bool ssm_map(SsmEncodeFn fn, CUtensorMap *m, const void *p, int B, int N, int K, int w, long long ld) {
    const cuuint64_t dims[4] = {(cuuint64_t)w, (cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)w * 2, (cuuint64_t)ld * 2, (cuuint64_t)N * ld * 2};
    const cuuint32_t box[4] = {64, 1, SQ, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Segments: the split that the two launches' chunk counts per SM favour.
void ssm_chunk_segments(int B, int H, int N, int d, int M, int num_sms, int &seg, int &segs) {
    const int nch = (N + SQ - 1) / SQ, dp = d <= 64 ? 64 : 128;
    const long long units = (long long)B * H * ((d + dp - 1) / dp), slots = (long long)num_sms * (M <= 64 ? 2 : 1);
    double best = 0;
    int pick = 1;
    for (int s = 1; s <= nch && s <= 64; ++s) {
        const int per = (nch + s - 1) / s, real = (nch + per - 1) / per;
        if (real != s) continue;
        const double main_waves = (double)((units * s + slots - 1) / slots);
        const double state_waves = s > 1 ? (double)((units * (s - 1) + 3 * num_sms - 1) / (3 * num_sms)) : 0.0;
        const double cost = main_waves * (per * 2.5 + 3.0 + 0.3 * (s - 1)) + state_waves * (per * 1.5 + 3.0);
        if (s == 1 || cost < best) {
            best = cost;
            pick = s;
        }
    }
    seg = (nch + pick - 1) / pick * SQ;
    segs = (N + seg - 1) / seg;
}

size_t ssm_chunk_workspace_bytes(int B, int H, int N, int d, int M, int num_sms) {
    int seg, segs;
    ssm_chunk_segments(B, H, N, d, M, num_sms, seg, segs);
    return segs < 2 ? 0 : (size_t)B * H * segs * ((size_t)M * d + 4) * sizeof(float);
}

template <int DP, int MP>
static ida_status launch_chunk(const ScanArgs &a, const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mc,
                               const CUtensorMap &my, cudaStream_t st) {
    constexpr int s_state = SsmSmem<DP, MP, true>::TOTAL, s_main = SsmSmem<DP, MP, false>::TOTAL;
    static_assert(s_main <= (MP == 64 ? 113 : 227) * 1024 && s_state <= 227 * 1024, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(ssm_chunk_kernel<DP, MP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, s_main);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ssm_chunk_kernel<DP, MP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, s_state);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long units = (long long)a.B * a.H * ((a.d + DP - 1) / DP);
    if (units * a.segs > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows and heads");
    if (a.segs > 1) {
        ssm_chunk_kernel<DP, MP, true><<<(unsigned)(units * (a.segs - 1)), STH, s_state, st>>>(a, mx, mb, mc, my);
        const ida_status s = launched("ssm segment states");
        if (s != IDA_OK) return s;
    }
    ssm_chunk_kernel<DP, MP, false><<<(unsigned)(units * a.segs), STH, s_main, st>>>(a, mx, mb, mc, my);
    return launched("ssm scan");
}

ida_status launch_ssm_chunk(const ScanArgs &a, cudaStream_t st) {
    const SsmEncodeFn fn = ssm_encode_fn();
    if (!fn) return fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    CUtensorMap mx, mb, mc, my;
    if (!ssm_map(fn, &mx, a.x, a.B, a.N, a.H, a.d, a.ldx) || !ssm_map(fn, &mb, a.b, a.B, a.N, a.G, a.M, a.ldb) ||
        !ssm_map(fn, &mc, a.c, a.B, a.N, a.G, a.M, a.ldc) ||
        !ssm_map(fn, &my, a.y, a.B, a.N, a.H, a.d, (long long)a.H * a.d))
        return fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    if (a.d <= 64)
        return a.M <= 64 ? launch_chunk<64, 64>(a, mx, mb, mc, my, st) : launch_chunk<64, 128>(a, mx, mb, mc, my, st);
    return a.M <= 64 ? launch_chunk<128, 64>(a, mx, mb, mc, my, st) : launch_chunk<128, 128>(a, mx, mb, mc, my, st);
}

}  // namespace ida
