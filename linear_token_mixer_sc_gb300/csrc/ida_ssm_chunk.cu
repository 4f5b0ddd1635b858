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
// Precision.  Everything accumulates in fp32.  P, c 2^S, the X_0 operand and, where only y comes
// of it, the scaled b are rounded to bf16 (each 2^-9 of a term on average, below y's own
// rounding).  States that leave the kernel (the final state, and a segment's last state, which the
// next one starts from) are fp32 results: for them the scaled b is kept as the sum of three bf16
// tiles, all 24 bits.  S is summed in 2^-32 fixed point: it is exact over any chunk or segment.
//
// One CTA of 256 threads walks the chunks of one (row, head, up to 128 channels, segment).  x, b
// and c tiles arrive by TMA with the 128-byte swizzle that the MMA descriptors name, so one copy
// serves as a K-major operand (b, c in G) and as an MN-major one (x, b in the state update, whose K
// is the position).  P is an A operand in TMEM: thread t of a lane quarter makes row t of it from
// row t of G.  The state stays in TMEM; y leaves through shared memory that is dead by then, by TMA.
// With M <= 64 two CTAs share an SM (256 TMEM columns and 75 or 101 KB each) and fill each other's
// waits: a chunk is a chain of copy, MMA, CUDA-core stage, MMA, epilogue.  The lower triangle gives
// the lane quarters of P 1 to 4 blocks of columns per warp; the scaling of b and c is dealt out so
// that all warps have the same total.
//
// Few (row, head) units do not fill the SMs: sequences are cut into segments.  A first launch
// (ssm_state_kernel: x and b only) leaves each segment's last state from zero, a second the states
// the segments start from, and the final state.  The state kernel walks a segment backwards, where
// the decay from a position to the segment's end is known without a look ahead, so its MMAs only
// accumulate and the copies and the scaling of the next chunk run beside them.
//
// Every wait is bounded.  On a timeout all threads of the CTA leave the loop together, the kernel
// records kErrWaitTimeout, waits (bounded) for its copy in flight, frees its TMEM and returns.
#include <mutex>

#include "ida_ssm_tc.cuh"

namespace ida {

using namespace tc;

constexpr int STH = 256;  // threads per CTA

// Shared memory map; DP, MP: channels and state rows rounded up to 64 or 128.
constexpr int SARR = 5 * SQ + 16;  // floats of one chunk's arrays (StepArrays)
template <int DP, int MP>
struct SsmSmem {
    static constexpr int X = 0;                            // [DP / 64][128 s][64] bf16
    static constexpr int B = X + DP / 64 * SSLAB;          // [MP / 64][128 s][64]: b, then scaled
    static constexpr int C = B + MP / 64 * SSLAB;          // [MP / 64][128 t][64]: c, then scaled
    static constexpr int SBS = DP * 128;                   // bytes of one slab of SB
    static constexpr int SB = C + MP / 64 * SSLAB;         // [MP / 64][DP j][64]: X_0^T
    // the output tile [DP / 64][128 t][64]: over SB, and a slab of its own where SB is smaller
    static constexpr int SB_BYTES = MP / 64 * SBS, OUT_BYTES = DP / 64 * SSLAB;
    static constexpr int OUT0 = DP == 64 && MP == 64 ? SB + SB_BYTES : SB;
    static constexpr int OUT1 = SB + SSLAB;
    static constexpr int MISC = OUT_BYTES > SB_BYTES ? SB + SB_BYTES + SSLAB : SB + SB_BYTES;
    static constexpr int ARR = MISC + 64;                  // two chunks' arrays
    static constexpr int TOT = ARR + 2 * SARR * 4;         // 4 64-bit totals
    static constexpr int TOTAL = TOT + 32;
};
// PARTS: bf16 tiles that the scaled b is kept in.  With one, two chunks are in flight.
template <int DP, int MP, int PARTS>
struct SsmStateSmem {
    static constexpr int NB = PARTS == 1 ? 2 : 1;
    static constexpr int X = 0;                            // [NB][DP / 64][128 s][64] bf16
    static constexpr int XB = DP / 64 * SSLAB, BB = MP / 64 * SSLAB * PARTS;
    static constexpr int B = X + NB * XB;                  // [NB][PARTS][MP / 64][128 s][64]
    static constexpr int MISC = B + NB * BB;
    static constexpr int ARR = MISC + 64;                  // two chunks' weights
    static constexpr int TOT = ARR + 2 * SQ * 4;
    static constexpr int TOTAL = TOT + 32;
};

template <int DP, int MP>
struct SsmTmem {
    static constexpr uint32_t G = 0;    // [t][s], later Y [t][j]
    static constexpr uint32_t P = 128;  // [t][s] bf16 pairs
    static constexpr uint32_t S = 192;  // [j][m]; with DP = 64 lanes 64.. repeat 0..63
    static constexpr uint32_t COLS = MP == 64 ? 256 : 512;
};

// What a chunk's step sizes give, for the positions s of the chunk.
struct StepArrays {
    float *cumf;  // S_s
    float *uf;    // S_s - log2 D_s
    float *rs;    // 2^(S at the end of s's block of 16 - uf)
    float *wst;   // 2^(S_Q - S_s) D_s
    float *et;    // 2^S_s
    float *cref;  // S at the end of each block of 16; [8]: 2^S_Q
    __device__ __forceinline__ StepArrays(float *p)
        : cumf(p), uf(p + SQ), rs(p + 2 * SQ), wst(p + 3 * SQ), et(p + 4 * SQ), cref(p + 5 * SQ) {}
};

template <int DP, int MP>
__global__ void __launch_bounds__(STH, MP == 64 ? 2 : 1)
    ssm_chunk_kernel(ScanArgs a, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y) {
    using L = SsmSmem<DP, MP>;
    using T = SsmTmem<DP, MP>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);  // 0 copies, 1 G, 2 Y, 3 state
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 48);
    float *arrays = reinterpret_cast<float *>(sm + L::ARR);
    long long *tot = reinterpret_cast<long long *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int q4 = warp & 3, half = warp >> 2, tl = 32 * q4 + lane;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d;
    const int slices = (d + DP - 1) / DP;
    int id = blockIdx.x;
    const int seg = id % a.segs;
    id /= a.segs;
    const int j0 = id % slices * DP, unit = id / slices, b = unit / H, h = unit % H, g = h / (H / a.G);
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg), nch = (t_end - t_begin + SQ - 1) / SQ;
    const __nv_bfloat16 *gdt = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)b * N * a.lddt + h;
    const float dt_bias = a.dt_bias[h], skip = a.D[h];
    const double rate2 = log2_rate(a.a_log[h]);
    constexpr uint32_t TILE_BYTES = (uint32_t)SSLAB * (DP / 64 + 2 * (MP / 64));

    if ((s0 & 1023u) != 0u) {  // the swizzle repeats every 1024 bytes
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_c);
        tma_prefetch_desc(&tm_y);
    }
    if (warp == 0) {
        tmem_alloc(tslot, T::COLS);
        tmem_relinquish();
    }
    const auto fetch = [&](int t0) {  // one thread
        mbar_arrive_expect_tx(&bar[0], TILE_BYTES);
#pragma unroll
        for (int i = 0; i < MP / 64; ++i) {
            tma_load_4d(sm + L::B + i * SSLAB, &tm_b, 64 * i, g, t0, b, &bar[0]);
            tma_load_4d(sm + L::C + i * SSLAB, &tm_c, 64 * i, g, t0, b, &bar[0]);
        }
#pragma unroll
        for (int i = 0; i < DP / 64; ++i) tma_load_4d(sm + L::X + i * SSLAB, &tm_x, j0 + 64 * i, h, t0, b, &bar[0]);
    };
    // the arrays of the chunk at t0, by warps 4 .. 7, into buffer `buf`; its raw steps were read before
    float dt_next = 0.f;
    const auto fetch_dt = [&](int t0) {
        const int k = tid - SQ;
        if (k >= 0) dt_next = t0 + k < t_end ? __bfloat162float(gdt[(size_t)(t0 + k) * a.lddt]) : 0.f;
    };
    const auto make_arrays = [&](int t0, int buf) {
        const int k = tid - SQ;
        if (k < 0) return;
        float delta = 0.f;
        if (t0 + k < t_end) delta = softplus(dt_next + dt_bias);  // behind the end nothing decays or is added
        long long all;
        const long long fx = chunk_sum(rate2, delta, k, tot, all);
        const StepArrays A(arrays + buf * SARR);
        const float s = (float)fx * kUnfix, u = s - log2f(delta);  // D = 0: +inf, and 2^(.. - u) = 0
        const float ref = __shfl_sync(0xffffffffu, s, lane | 15);
        A.cumf[k] = s;
        A.uf[k] = u;
        A.rs[k] = ex2(ref - u);
        A.wst[k] = ex2((float)(all - fx) * kUnfix) * delta;
        A.et[k] = ex2(s);
        if ((lane & 15) == 15) A.cref[k >> 4] = s;
        if (k == 0) A.cref[8] = ex2((float)all * kUnfix);
    };
    fetch_dt(t_begin);
    __syncthreads();
    if (tid == 0) fetch(t_begin);
    make_arrays(t_begin, 0);
    fetch_dt(t_begin + SQ);
    tc_fence_after();
    const uint32_t tm = *tslot;
    constexpr int MH = MP / 2;  // state rows of a warp half
    {
        // the state before the segment
        const int ch = DP == 64 ? (tl & 63) : tl;  // my channel; with DP = 64 lanes 64.. repeat 0..63
        const float *p = a.segs > 1 ? a.seg_state + ((size_t)unit * a.segs + seg) * M * d
                                    : (a.state_in ? a.state_in + (size_t)unit * M * d : nullptr);
        const bool mine = p && j0 + ch < d;
#pragma unroll
        for (int blk = 0; blk < MH / 16; ++blk) {
            const int m0 = half * MH + 16 * blk;
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                v[e] = mine && m0 + e < M ? __ldg(p + (size_t)(m0 + e) * d + j0 + ch) : 0.f;
            tmem_st16(tm + lane_base + T::S + m0, v);
        }
        tmem_wait_st();
    }
    bool ok = true;
    int i = 0;
    for (; i < nch; ++i) {
        const int t0 = t_begin + i * SQ;
        const uint32_t par = i & 1;
        const StepArrays A(arrays + par * SARR);
        ok = mbar_wait(&bar[0], par) && ok;
        if (__syncthreads_or(!ok)) break;  // the tiles and this chunk's arrays are there, the last state update is done
        tc_fence_after();
        if (warp == 0 && elect_one()) {
            const SmemDesc da = sw_desc(s0 + L::C, 16), db = sw_desc(s0 + L::B, 16);
            constexpr uint32_t id_g = idesc(128, 128, 1, 1);
#pragma unroll
            for (int k = 0; k < MP / 16; ++k) {
                const uint32_t off = (k / 4) * SSLAB + (k % 4) * 32;
                mma_f16(tm + T::G, sw_step(da, off), sw_step(db, off), id_g, k > 0);
            }
            mma_commit(&bar[1]);
        }
        __syncwarp();
        // the state: its bf16 copy for Y, kept until SB is free, and its decay over the chunk
        uint32_t sb[MH / 2];
        const float decay = A.cref[8];
#pragma unroll
        for (int blk = 0; blk < MH / 32; ++blk) {
            const uint32_t at = tm + lane_base + T::S + half * MH + 32 * blk;
            float v[32];
            tmem_ld16(at, v);
            tmem_ld16(at + 16, v + 16);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) sb[16 * blk + e] = pack_bf16(v[2 * e], v[2 * e + 1]);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= decay;
            tmem_st16(at, v);
            tmem_st16(at + 16, v + 16);
        }
        if (tid == 0) bulk_wait_read_all();  // y of the last chunk has left shared memory
        ok = mbar_wait(&bar[1], par);
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (tl < DP)
#pragma unroll
            for (int c = 0; c < MH / 8; ++c) {
                const int p = half * (MH / 8) + c;  // 16-byte piece of row tl
                *reinterpret_cast<uint4 *>(sm + L::SB + p / 8 * L::SBS + sw_off(tl, p % 8)) =
                    make_uint4(sb[4 * c], sb[4 * c + 1], sb[4 * c + 2], sb[4 * c + 3]);
            }
        {
            // P: row tl; the two warps of a lane quarter take blocks of 16 columns in turn
            const float ct = A.cumf[tl];
            for (int kb = half; kb < 8; kb += 2) {
                uint32_t w[8];
                if (kb > 2 * q4 + 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                } else {
                    float v[16];
                    tmem_ld16(tm + lane_base + T::G + 16 * kb, v);
                    if (kb < 2 * q4) {  // wholly before my rows: one exponential for the block
                        const float f = ex2(ct - A.cref[kb]);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 r = *reinterpret_cast<const float4 *>(A.rs + 16 * kb + e);
                            v[e] *= f * r.x;
                            v[e + 1] *= f * r.y;
                            v[e + 2] *= f * r.z;
                            v[e + 3] *= f * r.w;
                        }
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int s = 16 * kb + e;
                            const float p = v[e] * ex2(ct - A.uf[s]);
                            v[e] = s < tl ? p : s == tl ? p + skip : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                }
                tmem_st8(tm + lane_base + T::P + 8 * kb, w);
            }
        }
        {
            // b 2^(S_Q - S_s) D_s and c 2^S_t, in units of 16 bytes of 32 rows: a block of P is worth
            // four of them, and a warp of lane quarter q has q + 1 blocks
            constexpr int UNITS = 2 * 4 * (MP / 8), BASE = UNITS / 8 + 6;
            const int n = BASE - 4 * q4, first = 2 * (BASE * q4 - 2 * q4 * (q4 - 1)) + half * n;
            // (n is even: two units' loads at a time)
            for (int k0 = first; k0 < first + n; k0 += 2) {
                uint4 *at[2], u[2];
                float f[2];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int k = k0 + o, r = 32 * (k & 3) + lane, p = (k >> 2) % (MP / 8);
                    const bool is_c = (k >> 2) >= MP / 8;
                    f[o] = is_c ? A.et[r] : A.wst[r];
                    at[o] = reinterpret_cast<uint4 *>(sm + (is_c ? L::C : L::B) + p / 8 * SSLAB + sw_off(r, p % 8));
                    u[o] = *at[o];
                }
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    float v[8];
                    Vec16<__nv_bfloat16>::unpack(u[o], v);
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] *= f[o];
                    *at[o] = Vec16<__nv_bfloat16>::pack(v);
                }
            }
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const SmemDesc dx = sw_desc(s0 + L::X, SSLAB);  // [K = s][j]
            constexpr uint32_t id_p = idesc(128, DP, 1, 1, 0, 1), id_s = idesc(128, DP, 1, 1);
#pragma unroll
            for (int k = 0; k < SQ / 16; ++k)
                mma_f16_t(tm + T::G, tm + T::P + 8 * k, sw_step(dx, k * 2048), id_p, k > 0);
            const SmemDesc dc = sw_desc(s0 + L::C, 16), ds = sw_desc(s0 + L::SB, 16);
#pragma unroll
            for (int k = 0; k < MP / 16; ++k)
                mma_f16(tm + T::G, sw_step(dc, k / 4 * SSLAB + k % 4 * 32), sw_step(ds, k / 4 * L::SBS + k % 4 * 32),
                        id_s, 1);
            mma_commit(&bar[2]);
            // x^T as A: with DP = 64 its second 64 rows repeat the first
            const SmemDesc da = sw_desc(s0 + L::X, DP == 64 ? 0 : SSLAB), dh = sw_desc(s0 + L::B, SSLAB);
            constexpr uint32_t id_x = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll
            for (int k = 0; k < SQ / 16; ++k) mma_f16(tm + T::S, sw_step(da, k * 2048), sw_step(dh, k * 2048), id_x, 1);
            mma_commit(&bar[3]);
        }
        __syncwarp();
        if (i + 1 < nch) {
            make_arrays(t0 + SQ, par ^ 1);
            fetch_dt(t0 + 2 * SQ);
        }
        ok = mbar_wait(&bar[2], par);
        tc_fence_after();
        // y: row tl, half of the channels
        constexpr int CW = DP / 2;  // channels of a warp
        unsigned char *out = sm + (DP == 128 && half ? L::OUT1 : L::OUT0);
        const int p0 = DP == 128 ? 0 : half * 4;
#pragma unroll
        for (int blk = 0; blk < CW / 32; ++blk) {
            float v[32];
            tmem_ld16(tm + lane_base + T::G + half * CW + 32 * blk, v);
            tmem_ld16(tm + lane_base + T::G + half * CW + 32 * blk + 16, v + 16);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4 *>(out + sw_off(tl, p0 + 4 * blk + c)) = Vec16<__nv_bfloat16>::pack(v + 8 * c);
        }
        tc_fence_before();
        fence_proxy_async_smem();
        ok = mbar_wait(&bar[3], par) && ok;
        if (__syncthreads_or(!ok)) break;
        if (tid == 0) {
            if (i + 1 < nch) fetch(t0 + SQ);
#pragma unroll
            for (int s = 0; s < DP / 64; ++s)
                if (j0 + 64 * s < d) tma_store_4d(&tm_y, j0 + 64 * s, h, t0, b, sm + (s ? L::OUT1 : L::OUT0));
            bulk_commit();
        }
    }
    if (i < nch && tid == 0) {  // a wait ran out
        report_error(a.err, kErrWaitTimeout);
        mbar_wait(&bar[0], i & 1);  // the copy of this chunk, if it is still in flight
    }
    if (tid == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, T::COLS);
    }
}

// A segment's last state from zero (the first segment's: from state_in) and its log2 decay; a
// single segment's is the final state.  Chunks from the last to the first.  REV: what a segment
// passes on of its own adjoint, sum_t a_first .. a_t c_t dy_t^T, from dy and c in the places of x
// and b; there the sum up to a chunk is needed, so chunks go from the first to the last.
template <int DP, int MP, int PARTS, bool REV>
__global__ void __launch_bounds__(STH, MP == 64 ? 2 : 1)
    ssm_state_kernel(ScanArgs a, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b) {
    using L = SsmStateSmem<DP, MP, PARTS>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);  // 0, 1 copies, 2, 3 MMAs, of each buffer
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 48);
    float *arrays = reinterpret_cast<float *>(sm + L::ARR);
    long long *tot = reinterpret_cast<long long *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int q4 = warp & 3, half = warp >> 2, tl = 32 * q4 + lane;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d;
    const int slices = (d + DP - 1) / DP;
    int id = blockIdx.x;
    const int seg = id % a.state_segs;
    id /= a.state_segs;
    const int j0 = id % slices * DP, unit = id / slices, b = unit / H, h = unit % H, g = h / (H / a.G);
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg), nch = (t_end - t_begin + SQ - 1) / SQ;
    const __nv_bfloat16 *gdt = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)b * N * a.lddt + h;
    const float dt_bias = a.dt_bias[h];
    const double rate2 = log2_rate(a.a_log[h]);

    if ((s0 & 1023u) != 0u) {
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_b);
    }
    if (warp == 0) {
        tmem_alloc(tslot, MP);
        tmem_relinquish();
    }
    const auto start_of = [&](int n) { return t_begin + (REV ? n : nch - 1 - n) * SQ; };  // the n-th chunk walked
    const auto fetch = [&](int n) {  // one thread
        const int buf = n % L::NB, t0 = start_of(n);
        mbar_arrive_expect_tx(&bar[buf], (uint32_t)SSLAB * (DP / 64 + MP / 64));
#pragma unroll
        for (int i = 0; i < MP / 64; ++i)
            tma_load_4d(sm + L::B + buf * L::BB + i * SSLAB, &tm_b, 64 * i, g, t0, b, &bar[buf]);
#pragma unroll
        for (int i = 0; i < DP / 64; ++i)
            tma_load_4d(sm + L::X + buf * L::XB + i * SSLAB, &tm_x, j0 + 64 * i, h, t0, b, &bar[buf]);
    };
    float dt_next = 0.f;
    const auto fetch_dt = [&](int n) {
        const int k = tid - SQ, p = start_of(n) + k;
        if (k >= 0) dt_next = n < nch && p < t_end ? __bfloat162float(gdt[(size_t)p * a.lddt]) : 0.f;
    };
    long long behind = 0;  // log2 a summed over the chunks done, in warps 4 .. 7
    const auto make_weights = [&](int n) {
        const int k = tid - SQ;
        if (k < 0) return;
        float delta = 0.f;
        if (start_of(n) + k < t_end) delta = softplus(dt_next + dt_bias);
        long long all;
        const long long fx = chunk_sum(rate2, delta, k, tot, all);
        arrays[(n & 1) * SQ + k] = REV ? (start_of(n) + k < t_end ? ex2_fix(fx + behind) : 0.f) : ex2_fix(all - fx + behind) * delta;
        behind += all;
    };
    fetch_dt(0);
    __syncthreads();
    if (tid == 0)
        for (int n = 0; n < L::NB && n < nch; ++n) fetch(n);
    make_weights(0);
    fetch_dt(1);
    tc_fence_after();
    const uint32_t tm = *tslot;
    bool ok = true;
    int n = 0;
    for (; n < nch; ++n) {
        const int buf = n % L::NB;
        const uint32_t par = (n / L::NB) & 1;
        ok = mbar_wait(&bar[buf], par) && ok;
        if (__syncthreads_or(!ok)) break;  // the tiles and the weights are there
        // b 2^(S_end - S_s) D_s: row r, half of the columns
        const int r = tid & 127, p0 = (tid >> 7) * (MP / 16);
        const float w = arrays[(n & 1) * SQ + r];
#pragma unroll
        for (int k = 0; k < MP / 16; ++k) {
            const int p = p0 + k;
            unsigned char *at = sm + L::B + buf * L::BB + p / 8 * SSLAB + sw_off(r, p % 8);
            float v[8];
            Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<uint4 *>(at), v);
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] *= w;
            uint4 u = Vec16<__nv_bfloat16>::pack(v);
            *reinterpret_cast<uint4 *>(at) = u;
#pragma unroll
            for (int part = 1; part < PARTS; ++part) {  // what the rounding dropped
                float hi[8];
                Vec16<__nv_bfloat16>::unpack(u, hi);
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] -= hi[x];
                u = Vec16<__nv_bfloat16>::pack(v);
                *reinterpret_cast<uint4 *>(at + part * (MP / 64) * SSLAB) = u;
            }
        }
        fence_proxy_async_smem();
        // two buffers: the other one's next copy, once its MMAs, issued before this scaling, have read it
        if (L::NB == 2 && tid == 0 && n > 0 && n + 1 < nch) {
            ok = mbar_wait(&bar[2 + (buf ^ 1)], ((n - 1) / 2) & 1);
            if (ok) fetch(n + 1);
        }
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            // x^T as A: with DP = 64 its second 64 rows repeat the first
            const SmemDesc da = sw_desc(s0 + L::X + buf * L::XB, DP == 64 ? 0 : SSLAB);
            constexpr uint32_t id_x = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part) {  // the small parts first: fewer roundings of the large sum
                const SmemDesc dh = sw_desc(s0 + L::B + buf * L::BB + part * (MP / 64) * SSLAB, SSLAB);
#pragma unroll
                for (int k = 0; k < SQ / 16; ++k)
                    mma_f16(tm, sw_step(da, k * 2048), sw_step(dh, k * 2048), id_x, n > 0 || part < PARTS - 1 || k > 0);
            }
            mma_commit(&bar[2 + buf]);
        }
        __syncwarp();
        if (n + 1 < nch) {
            make_weights(n + 1);
            fetch_dt(n + 2);
        }
        if (L::NB == 1 && tid == 0 && n + 1 < nch) {
            ok = mbar_wait(&bar[2], par);
            if (ok) fetch(n + 1);
        }
    }
    if (n == nch) {
        for (int k = 0; k < L::NB && k < nch; ++k) {  // the last MMAs of each buffer
            const int last = nch - 1 - k;
            ok = mbar_wait(&bar[2 + last % L::NB], (last / L::NB) & 1) && ok;
        }
    }
    tc_fence_after();
    if (__syncthreads_or(!ok)) {  // a wait ran out
        if (tid == 0) {
            report_error(a.err, kErrWaitTimeout);
            for (int k = 0; k < L::NB && n + k < nch; ++k) mbar_wait(&bar[(n + k) % L::NB], ((n + k) / L::NB) & 1);
        }
    } else {
        // a single segment's last state is the final state
        float *out = a.segs == 1 && a.final_state ? a.final_state + (size_t)unit * M * d
                                                  : a.seg_state + ((size_t)unit * a.segs + seg) * M * d;
        if (tid >= SQ && tid < SQ + 1) arrays[0] = (float)behind * kUnfix;
        __syncthreads();
        const float *in = !REV && seg == 0 && a.state_in ? a.state_in + (size_t)unit * M * d : nullptr;
        const float total = arrays[0], f = ex2(total);
        constexpr int MH = MP / 2;
        if (DP == 128 || tl < DP) {
#pragma unroll
            for (int blk = 0; blk < MH / 16; ++blk) {
                const int m0 = half * MH + 16 * blk;
                float v[16];
                tmem_ld16(tm + lane_base + m0, v);
                tmem_wait_ld();
                if (j0 + tl < d)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (m0 + e < M) {
                            const size_t at = (size_t)(m0 + e) * d + j0 + tl;
                            out[at] = in ? fmaf(f, __ldg(in + at), v[e]) : v[e];
                        }
            }
        }
        if (!REV && tid == 0 && j0 == 0 && a.segs > 1) a.seg_log[(size_t)unit * a.segs + seg] = total;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, MP);
    }
}

// Segment states, in place: seg_state[s] becomes the state before segment s; the final state where
// it is wanted.  One thread per four state elements.
__global__ void __launch_bounds__(256) ssm_carry_kernel(ScanArgs a) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int n = a.M * a.d / 4;
    const int unit = (int)(i / n), e = (int)(i % n);
    if (unit >= a.B * a.H) return;
    float4 *p = reinterpret_cast<float4 *>(a.seg_state + (size_t)unit * a.segs * a.M * a.d) + e;
    const float *lg = a.seg_log + (size_t)unit * a.segs;
    float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
    // the first segment starts from the given state, which its last state holds
    float4 start = X;
    if (a.state_in) start = __ldg(reinterpret_cast<const float4 *>(a.state_in + (size_t)unit * a.M * a.d) + e);
    constexpr int K = 8;
    for (int s0 = 0; s0 < a.segs; s0 += K) {
        float4 v[K];
        float f[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (s0 + k < a.state_segs) {
                v[k] = p[(size_t)(s0 + k) * n];
                f[k] = lg[s0 + k];
            }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int s = s0 + k;
            if (s >= a.segs) break;
            p[(size_t)s * n] = s == 0 ? start : X;
            if (s < a.state_segs) {
                const float w = ex2(f[k]);
                X = make_float4(fmaf(w, X.x, v[k].x), fmaf(w, X.y, v[k].y), fmaf(w, X.z, v[k].z), fmaf(w, X.w, v[k].w));
            }
        }
    }
    if (a.final_state) reinterpret_cast<float4 *>(a.final_state + (size_t)unit * a.M * a.d)[e] = X;
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

ida_status ssm_map(CUtensorMap *m, const void *p, int B, int N, int K, int w, long long ld, int rows) {
    const SsmEncodeFn fn = ssm_encode_fn();
    if (!fn) return fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[4] = {(cuuint64_t)w, (cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)w * 2, (cuuint64_t)ld * 2, (cuuint64_t)N * ld * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? IDA_OK : fail_with(IDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
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
        const double state_waves = s > 1 ? (double)((units * (s - 1) + 2 * num_sms - 1) / (2 * num_sms)) : 0.0;
        const double cost = main_waves * (per * 3.4 + 3.0) + (s > 1 ? state_waves * (per * 1.5 + 3.0) + 4.0 : 0.0);
        if (s == 1 || cost < best) {
            best = cost;
            pick = s;
        }
    }
    seg = (nch + pick - 1) / pick * SQ;
    segs = (N + seg - 1) / seg;
}

template <int DP, int MP, int PARTS, bool REV>
static ida_status launch_states(const ScanArgs &a, cudaStream_t st) {
    constexpr int smem = SsmStateSmem<DP, MP, PARTS>::TOTAL;
    static_assert(smem <= (MP == 64 ? 113 : 227) * 1024, "shared memory budget");
    CUtensorMap mx, mb;
    ida_status s = ssm_map(&mx, a.x, a.B, a.N, a.H, a.d, a.ldx);
    if (s == IDA_OK) s = ssm_map(&mb, a.b, a.B, a.N, a.G, a.M, a.ldb);
    if (s != IDA_OK) return s;
    const auto kernel = ssm_state_kernel<DP, MP, PARTS, REV>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long units = (long long)a.B * a.H * ((a.d + DP - 1) / DP);
    kernel<<<(unsigned)(units * a.state_segs), STH, smem, st>>>(a, mx, mb);
    return launched("ssm segment states");
}

template <int DP, int MP>
static ida_status launch_states_of(const ScanArgs &a, bool exact, bool rev, cudaStream_t st) {
    if (rev) return launch_states<DP, MP, 3, true>(a, st);
    return exact ? launch_states<DP, MP, 3, false>(a, st) : launch_states<DP, MP, 1, false>(a, st);
}

ida_status launch_ssm_states(const ScanArgs &a, bool exact, bool rev, cudaStream_t st) {
    if (a.d <= 64) return a.M <= 64 ? launch_states_of<64, 64>(a, exact, rev, st) : launch_states_of<64, 128>(a, exact, rev, st);
    return a.M <= 64 ? launch_states_of<128, 64>(a, exact, rev, st) : launch_states_of<128, 128>(a, exact, rev, st);
}

template <int DP, int MP>
static ida_status launch_chunk(const ScanArgs &a, const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mc,
                               const CUtensorMap &my, cudaStream_t st) {
    constexpr int smem = SsmSmem<DP, MP>::TOTAL;
    static_assert(smem <= (MP == 64 ? 113 : 227) * 1024, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(ssm_chunk_kernel<DP, MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long units = (long long)a.B * a.H * ((a.d + DP - 1) / DP);
    if (units * a.segs > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows and heads");
    ida_status s = IDA_OK;
    if (a.state_segs > 0) s = launch_ssm_states(a, a.final_state != nullptr, false, st);
    if (s == IDA_OK && a.segs > 1) {
        const long long n = (long long)a.B * a.H * (a.M * a.d / 4);
        ssm_carry_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
        s = launched("ssm segment sums");
    }
    if (s != IDA_OK) return s;
    ssm_chunk_kernel<DP, MP><<<(unsigned)(units * a.segs), STH, smem, st>>>(a, mx, mb, mc, my);
    return launched("ssm scan");
}

ida_status launch_ssm_chunk(const ScanArgs &a, cudaStream_t st) {
    CUtensorMap mx, mb, mc, my;
    ida_status s = ssm_map(&mx, a.x, a.B, a.N, a.H, a.d, a.ldx);
    if (s == IDA_OK) s = ssm_map(&mb, a.b, a.B, a.N, a.G, a.M, a.ldb);
    if (s == IDA_OK) s = ssm_map(&mc, a.c, a.B, a.N, a.G, a.M, a.ldc);
    if (s == IDA_OK) s = ssm_map(&my, a.y, a.B, a.N, a.H, a.d, (long long)a.H * a.d);
    if (s != IDA_OK) return s;
    if (a.d <= 64)
        return a.M <= 64 ? launch_chunk<64, 64>(a, mx, mb, mc, my, st) : launch_chunk<64, 128>(a, mx, mb, mc, my, st);
    return a.M <= 64 ? launch_chunk<128, 64>(a, mx, mb, mc, my, st) : launch_chunk<128, 128>(a, mx, mb, mc, my, st);
}

}  // namespace ida
