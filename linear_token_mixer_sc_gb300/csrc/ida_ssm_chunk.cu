// ida_ssm_chunk.cu -- the selective scan in chunks on the tcgen05 tensor cores (bf16 inputs).
//
// Over a chunk of Q = 128 positions, with S_t the sum of log2 a up to position t of it, X_0 the
// state before it and X_Q the state behind it (see ida_ssm.cuh for the recurrence):
//   G    [t][s]  = c_t . b_s                                   MMA, K = M
//   P    [t][s]  = G 2^(S_t - S_s) D_s (s <= t)                CUDA cores, G from TMEM, P to TMEM
//   Y    [t][j]  = P x + 2^S_t (c_t X_0) + D x_t               MMAs, K = Q and K = M
//   X_Q^T [j][m] = 2^S_Q X_0^T + x^T (b_s 2^(S_Q - S_s) D_s)   scaled in TMEM, then MMA, K = Q
// Decays are differences of S taken before the exponential, so no weight but D_s exceeds 1.  (Where a block
// of 16 positions holds the diagonal, a weight is the product of a factor up to 2^64 and one as small.)
//
// Precision.  Everything accumulates in fp32.  P, the X_0 operand and the chunk kernel's scaled b are
// rounded to bf16 (each 2^-9 of a term on average, as y's own rounding); c is not: 2^S_t scales the rows
// of c X_0.  The states that a segment starts from and the final state are fp32 results, so that y is the
// same whether that one is wanted or not: for them the scaled b is kept as the sum of three bf16 tiles, all
// 24 bits, and S is summed in 2^-32 fixed point.  (Starting segments from one tile's sums: 55.9 us for 57.6
// at 4 x 4096, and another y.)  The chunk kernel sums it in two floats, one of them exactly: a position that
// forgets everything takes nothing from the decays behind it.  (One float and D in it as log2 D: y 3.4 times
// its error bound off behind a step size of 1e5, 17 times with rates of e^9 and step sizes of 10; fixed
// point: 2.46 us a chunk for 2.26.)
//
// One CTA per SM walks the chunks of one (row, head, up to 128 channels, segment), its warps in
// roles that hand chunks on through mbarriers, so that a chunk's copy, MMAs, CUDA-core stages and
// output overlap its neighbours':
//   warp 0      copies: x, b and c by TMA, two chunks ahead where shared memory allows
//   warp 1      issues all MMAs
//   warps 4-7   the step sizes' sums and exponentials, two chunks ahead; half of b scaled in place
//   warps 8-15  P: thread t of a lane quarter makes row t from row t of G, in G's own place in TMEM
//               (each half of a row is read and replaced by one warp), an A operand there
//   warps 16-23 the rows of (c X_0) in Y, half a row each, scaled by 2^S_t and D x
//               added, in fp32, before P x is; y out by TMA
//   warps 24-27 the other half of b; the state's bf16 copy for Y and its decay in TMEM
// What bounds it: the chain c X_0 - scaled rows - P x - state of a chunk, 4600 cycles, of which the MMAs'
// reads of shared memory are 2300.  4 x 4096 positions of 16 heads of 128 x 64: 36 us, 57.6 with the segment
// states before it.  Its warps run different code, so loops stay short: with all of them unrolled (66 KB)
// they waited for instructions, 60 us.  (All stages in one group of 256 threads, two CTAs per SM: 45 us for
// the 36, 8500 cycles a chunk, most of them waits for the next stage.  When the whole took 56 us: D as a part
// of P, rounded with it, 55, but y's error is 2.3e-3 of its size instead of 1.8e-3, 1.7e-3 of which are its own
// rounding; four warps for the rows, 58.)
// The tiles have the 128-byte swizzle that the MMA descriptors name, so one copy serves as a
// K-major operand (b, c in G) and as an MN-major one (x, b in the state update, whose K is the
// position).  The state stays in TMEM.
//
// Few (row, head) units do not fill the SMs: sequences are cut into segments.  A first launch
// (ssm_state_kernel: x and b only) leaves the last states from zero of parts of the segments, a
// second the states the segments start from, and the final state.  The state kernel walks a part
// backwards, where the decay from a position to the part's end is known without a look ahead, so its
// MMAs only accumulate and the next chunk's weights are made beside them.  (Its copy waits for them: three
// tiles of b leave room for one buffer with two CTAs an SM.)
//
// Every wait is bounded.  On a timeout the warps of a role leave their loop together (the others
// run out of waits of their own), the kernel records kErrWaitTimeout, waits (bounded) for its copies
// in flight, frees its TMEM and returns.
#include <mutex>

#include "ida_ssm_tc.cuh"

namespace ida {

using namespace tc;

constexpr int STH = 256;   // threads per CTA of the state kernel
constexpr int CTH = 896;   // threads per CTA of the chunk kernel

// The chunk kernel's mbarriers: those of chunk i, or of chunks i with the same i % 2.
enum {
    kFullBC = 0,   // [2] b and c are there
    kFreeBC = 2,   // [2] their buffer may be overwritten
    kFullX = 4,    // [2] x
    kFreeX = 6,    // [2]
    kG = 8,        // [2] G is complete
    kP = 10,       // [2] P is complete
    kY = 12,       // [2] Y is complete
    kScaled = 14,  // scaled b, the state's bf16 copy and its decay
    kState = 15,   // the state update is complete
    kCX = 16,      // c X_0 is complete
    kRows = 17,    // its rows are scaled
    kFreeY = 18,   // Y has been read
    kOut = 19,     // the output tile has left shared memory
    kArr = 20,     // [4] the chunk's arrays are there (of chunks with the same i % 4)
    kFreeArr = 24, // [4] and have been used
    kBars = 28
};

// Shared memory map; DP, MP: channels and state rows rounded up to 64 or 128.
constexpr int SARR = 6 * SQ + 32;  // floats of one chunk's arrays (StepArrays)
template <int DP, int MP>
struct SsmSmem {
    static constexpr int NX = DP == 128 && MP == 128 ? 1 : 2;  // buffers of x
    static constexpr int XB = DP / 64 * SSLAB, BB = MP / 64 * SSLAB;
    static constexpr int X = 0;                    // [NX][DP / 64][128 s][64] bf16
    static constexpr int B = X + NX * XB;          // [2][MP / 64][128 s][64]: b, then scaled
    static constexpr int C = B + 2 * BB;           // [2][MP / 64][128 t][64]
    static constexpr int SBS = DP * 128;           // bytes of one slab of SB
    static constexpr int SB = C + 2 * BB;          // [MP / 64][DP j][64]: X_0^T
    static constexpr bool OUT_OVER_SB = NX == 1;   // the output tile [DP / 64][128 t][64], where it does not fit beside SB
    static constexpr int OUT = OUT_OVER_SB ? SB : SB + MP / 64 * SBS;
    static constexpr int MISC = OUT + XB;
    static constexpr int ARR = MISC + 256;         // four chunks' arrays
    static constexpr int TOT = ARR + 4 * SARR * 4; // 4 totals
    static constexpr int TOTAL = TOT + 32;
};
constexpr int PARTS = 3;  // bf16 tiles that the state kernel keeps the scaled b in
template <int DP, int MP>
struct SsmStateSmem {
    static constexpr int X = 0;                            // [DP / 64][128 s][64] bf16
    static constexpr int B = X + DP / 64 * SSLAB;          // [PARTS][MP / 64][128 s][64]
    static constexpr int MISC = B + PARTS * (MP / 64) * SSLAB;
    static constexpr int ARR = MISC + 64;                  // two chunks' weights
    static constexpr int TOT = ARR + 2 * SQ * 4;
    static constexpr int TOTAL = TOT + 32;
};

// TMEM columns: G of two chunks ([t][s]; P of each in its place, bf16 pairs of s 64 h .. at 64 h ..),
// Y [t][j], the state [j][m] (with DP = 64 lanes 64.. repeat 0..63).
constexpr uint32_t TG = 0, TY = 256, TS = 384, TCOLS = 512;

// What a chunk's step sizes give, for the positions s of the chunk.  S is kept in two floats: a position
// that forgets everything leaves it large, and the small decays behind it are differences of it.
struct StepArrays {
    float *sh, *sl;        // S_s
    float *delta;          // D_s
    float *rs;             // 2^(S at the end of s's block of 16 - S_s) D_s
    float *et;             // 2^S_s
    float *wst;            // 2^(S_Q - S_s) D_s
    float *crefh, *crefl;  // S at the end of each block of 16
    float *span;           // how far S falls from the first to the last position of each block
    float *decay;          // 2^S_Q
    __device__ __forceinline__ StepArrays(float *p)
        : sh(p), sl(p + SQ), delta(p + 2 * SQ), rs(p + 3 * SQ), et(p + 4 * SQ), wst(p + 5 * SQ), crefh(p + 6 * SQ),
          crefl(p + 6 * SQ + 8), span(p + 6 * SQ + 16), decay(p + 6 * SQ + 24) {}
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// whether `p` holds in any of n threads, which all get the answer
__device__ __forceinline__ bool named_any(int id, int n, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)p)
        : "memory");
    return r != 0;
}

// Half of the 16-byte pieces of row r of b, from piece p0 on, scaled in place.
template <int MP>
__device__ __forceinline__ void scale_b(unsigned char *pb, int r, int p0, float weight) {
    constexpr int N = MP / 16;
    uint4 u[N];
#pragma unroll
    for (int p = 0; p < N; ++p) u[p] = *reinterpret_cast<uint4 *>(pb + (p0 + p) / 8 * SSLAB + sw_off(r, (p0 + p) % 8));
#pragma unroll
    for (int p = 0; p < N; ++p) {
        float v[8];
        Vec16<__nv_bfloat16>::unpack(u[p], v);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] *= weight;
        *reinterpret_cast<uint4 *>(pb + (p0 + p) / 8 * SSLAB + sw_off(r, (p0 + p) % 8)) = Vec16<__nv_bfloat16>::pack(v);
    }
}

template <int DP, int MP>
__global__ void __launch_bounds__(CTH, 1)
    ssm_chunk_kernel(ScanArgs a, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y) {
    using L = SsmSmem<DP, MP>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 8 * kBars);
    uint32_t *failed = tslot + 1;
    float *arrays = reinterpret_cast<float *>(sm + L::ARR);
    float2 *tot = reinterpret_cast<float2 *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int q4 = warp & 3, tl = 32 * q4 + lane;  // the lane quarter of TMEM this warp reaches, and its lane
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d;
    const int slices = (d + DP - 1) / DP;
    int id = blockIdx.x;
    const int seg = id % a.segs;
    id /= a.segs;
    const int j0 = id % slices * DP, unit = id / slices, b = unit / H, h = unit % H, g = h / (H / a.G);
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg), nch = (t_end - t_begin + SQ - 1) / SQ;

    if ((s0 & 1023u) != 0u) {  // the swizzle repeats every 1024 bytes
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i)
            mbar_init(&bar[i], i == kP || i == kP + 1 || i == kScaled || i == kRows || i == kFreeY ? 8 : i >= kArr && i < kFreeArr ? 4 : 1);
        fence_mbar_init();
        *failed = 0;
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_c);
        tma_prefetch_desc(&tm_y);
    }
    if (warp == 1) {
        tmem_alloc(tslot, TCOLS);
        tmem_relinquish();
    }
    dependent_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    const auto wait = [&](int k, uint32_t parity) { return mbar_wait(&bar[k], parity); };
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < nch && ok; ++i) {
                const int t0 = t_begin + i * SQ, c = i & 1, x = i % L::NX;
                if (i >= 2) ok = wait(kFreeBC + c, ((i >> 1) - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&bar[kFullBC + c], 2 * L::BB);
#pragma unroll
                for (int k = 0; k < MP / 64; ++k) {
                    tma_load_4d(sm + L::B + c * L::BB + k * SSLAB, &tm_b, 64 * k, g, t0, b, &bar[kFullBC + c]);
                    tma_load_4d(sm + L::C + c * L::BB + k * SSLAB, &tm_c, 64 * k, g, t0, b, &bar[kFullBC + c]);
                }
                if (i >= L::NX) ok = wait(kFreeX + x, (i / L::NX - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&bar[kFullX + x], L::XB);
#pragma unroll
                for (int k = 0; k < DP / 64; ++k)
                    tma_load_4d(sm + L::X + x * L::XB + k * SSLAB, &tm_x, j0 + 64 * k, h, t0, b, &bar[kFullX + x]);
            }
            if (!ok) {  // the copies in flight: this chunk's b and c, and the two before it
                wait(kFullBC + (i & 1), (i >> 1) & 1);
                if (i > 0) {
                    wait(kFullBC + ((i - 1) & 1), ((i - 1) >> 1) & 1);
                    wait(kFullX + (i - 1) % L::NX, ((i - 1) / L::NX) & 1);
                }
            }
        }
    } else if (warp == 1) {
        // all lanes wait, one issues: a uniform branch, which the MMAs' operands want (issued from a branch
        // on the lane they took three times as long)
        const auto issue_g = [&](int i) {
            const SmemDesc dc = sw_desc(s0 + L::C + (i & 1) * L::BB, 16), db = sw_desc(s0 + L::B + (i & 1) * L::BB, 16);
            constexpr uint32_t id_g = idesc(128, 128, 1, 1);
#pragma unroll
            for (int k = 0; k < MP / 16; ++k) {
                const uint32_t off = (k / 4) * SSLAB + (k % 4) * 32;
                mma_f16(tm + TG + 128 * (i & 1), sw_step(dc, off), sw_step(db, off), id_g, k > 0);
            }
            mma_commit(&bar[kG + (i & 1)]);
        };
        const auto all_wait = [&](int k, uint32_t parity) { return !__any_sync(0xffffffffu, !wait(k, parity)); };
        ok = all_wait(kFullBC, 0);
        if (ok && elect_one()) issue_g(0);
        for (int i = 0; i < nch && ok; ++i) {
            const int c = i & 1, x = i % L::NX;
            const uint32_t par = i & 1;
            ok = all_wait(kScaled, par) && all_wait(kFullX + x, (i / L::NX) & 1);
            if (!ok) break;
            if (elect_one()) {
                tc_fence_after();
                // x^T as A: with DP = 64 its second 64 rows repeat the first
                const SmemDesc da = sw_desc(s0 + L::X + x * L::XB, DP == 64 ? 0 : SSLAB);
                const SmemDesc dh = sw_desc(s0 + L::B + c * L::BB, SSLAB);
                constexpr uint32_t id_x = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll
                for (int k = 0; k < SQ / 16; ++k) mma_f16(tm + TS, sw_step(da, k * 2048), sw_step(dh, k * 2048), id_x, 1);
                mma_commit(&bar[kState]);
            }
            __syncwarp();
            if (i > 0) ok = all_wait(kFreeY, par ^ 1);
            if (!ok) break;
            if (elect_one()) {
                tc_fence_after();
                const SmemDesc dc = sw_desc(s0 + L::C + c * L::BB, 16), ds = sw_desc(s0 + L::SB, 16);
                constexpr uint32_t id_s = idesc(128, DP, 1, 1);
#pragma unroll
                for (int k = 0; k < MP / 16; ++k)
                    mma_f16(tm + TY, sw_step(dc, k / 4 * SSLAB + k % 4 * 32), sw_step(ds, k / 4 * L::SBS + k % 4 * 32), id_s, k > 0);
                mma_commit(&bar[kCX]);
                mma_commit(&bar[kFreeBC + c]);
            }
            __syncwarp();
            if (i + 1 < nch) {  // in the place of P of chunk i - 1, which the MMAs before have read
                ok = all_wait(kFullBC + (c ^ 1), ((i + 1) >> 1) & 1);
                if (!ok) break;
                if (elect_one()) issue_g(i + 1);
                __syncwarp();
            }
            ok = all_wait(kRows, par) && all_wait(kP + c, (i >> 1) & 1);
            if (!ok) break;
            if (elect_one()) {
                tc_fence_after();
                const SmemDesc dx = sw_desc(s0 + L::X + x * L::XB, SSLAB);  // [K = s][j]
                constexpr uint32_t id_p = idesc(128, DP, 1, 1, 0, 1);
#pragma unroll
                for (int k = 0; k < SQ / 16; ++k)
                    mma_f16_t(tm + TY, tm + TG + 128 * c + 64 * (k / 4) + 8 * (k % 4), sw_step(dx, k * 2048), id_p, 1);
                mma_commit(&bar[kY + c]);
                mma_commit(&bar[kFreeX + x]);
            }
            __syncwarp();
        }
    } else if (warp >= 4 && warp < 8) {
        const int k = tid - 128;  // position of the chunk
        const __nv_bfloat16 *gdt = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)b * N * a.lddt + h;
        const float dt_bias = a.dt_bias[h];
        const float rate2 = scan_rate(a.a_log[h]) * 1.4426950408889634f;
        const auto dt_of = [&](int i) {
            const int p = t_begin + i * SQ + k;
            return i < nch && p < t_end ? __bfloat162float(gdt[(size_t)p * a.lddt]) : 0.f;
        };
        float dt_next = dt_of(0);
        const auto make_arrays = [&](int i) {
            const float delta = t_begin + i * SQ + k < t_end ? softplus(dt_next + dt_bias) : 0.f;  // behind the end nothing decays or is added
            dt_next = dt_of(i + 1);
            if (i >= 4) ok = wait(kFreeArr + (i & 3), ((i >> 2) - 1) & 1);
            // log2 a in two floats, a multiple of 1/64 and the rest, summed apart: the sums of the first are exact
            // (2^-512 is 0 here, and 128 times 512 has 22 bits of 1/64), those of the rest stay below 1
            const float p = fminf(rate2 * delta, 512.f), m = (p + 196608.f) - 196608.f;
            float hi = -m, lo = m - p;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, hi, o), v = __shfl_up_sync(0xffffffffu, lo, o);
                if (lane >= o) {
                    hi += u;
                    lo += v;
                }
            }
            if (lane == 31) tot[q4] = make_float2(hi, lo);
            if (named_any(1, 128, !ok)) return false;
            float2 all = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w == q4) {
                    hi += all.x;
                    lo += all.y;
                }
                const float2 u = tot[w];
                all.x += u.x;
                all.y += u.y;
            }
            named_sync(1, 128);  // the totals have been read
            const StepArrays A(arrays + (i & 3) * SARR);
            const int end = lane | 15;  // of my block of 16
            const float rh = __shfl_sync(0xffffffffu, hi, end), rl = __shfl_sync(0xffffffffu, lo, end);
            const float first = __shfl_sync(0xffffffffu, hi, lane & 16);
            A.sh[k] = hi;
            A.sl[k] = lo;
            A.delta[k] = delta;
            A.rs[k] = ex2((rh - hi) + (rl - lo)) * delta;
            A.et[k] = ex2(hi + lo);
            A.wst[k] = ex2((all.x - hi) + (all.y - lo)) * delta;
            if ((lane & 15) == 15) {
                A.crefh[k >> 4] = hi;
                A.crefl[k >> 4] = lo;
                A.span[k >> 4] = first - hi;
            }
            if (k == 0) *A.decay = ex2(all.x + all.y);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kArr + (i & 3)]);
            return true;
        };
        bool go = make_arrays(0);
        if (go && nch > 1) go = make_arrays(1);
        for (int i = 0; i < nch && go; ++i) {
            const int c = i & 1;
            ok = wait(kFullBC + c, (i >> 1) & 1) && wait(kG + c, (i >> 1) & 1);  // G has read b
            if (named_any(1, 128, !ok)) {
                ok = false;
                break;
            }
            scale_b<MP>(sm + L::B + c * L::BB, k, MP / 16, StepArrays(arrays + (i & 3) * SARR).wst[k]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kScaled]);
            if (i + 2 < nch) go = make_arrays(i + 2);
        }
        if (!go) ok = false;
    } else if (warp >= 24) {
        const int k = tid - 768;  // row of b
        {
            // the state before the segment
            const int ch = DP == 64 ? (tl & 63) : tl;  // my channel; with DP = 64 lanes 64.. repeat 0..63
            const float *p = a.segs > 1 ? a.seg_state + ((size_t)unit * a.segs + seg) * a.fine * M * d
                                        : (a.state_in ? a.state_in + (size_t)unit * M * d : nullptr);
            const bool mine = p && j0 + ch < d;
#pragma unroll 1
            for (int m0 = 0; m0 < MP; m0 += 16) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = mine && m0 + e < M ? __ldcg(p + (size_t)(m0 + e) * d + j0 + ch) : 0.f;
                tmem_st16(tm + lane_base + TS + m0, v);
            }
            tmem_wait_st();
        }
        for (int i = 0; i < nch; ++i) {
            const int c = i & 1;
            const StepArrays A(arrays + (i & 3) * SARR);
            ok = wait(kArr + (i & 3), (i >> 2) & 1) && wait(kFullBC + c, (i >> 1) & 1) && wait(kG + c, (i >> 1) & 1);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            const float decay = *A.decay;
            scale_b<MP>(sm + L::B + c * L::BB, k, 0, A.wst[k]);
            if (i > 0) ok = wait(kState, (i - 1) & 1) && wait(kCX, (i - 1) & 1) && (!L::OUT_OVER_SB || wait(kOut, (i - 1) & 1));
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int m0 = 0; m0 < MP; m0 += 32) {
                const uint32_t at = tm + lane_base + TS + m0;
                float v[32];
                tmem_ld16(at, v);
                tmem_ld16(at + 16, v + 16);
                tmem_wait_ld();
                if (tl < DP)
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        *reinterpret_cast<uint4 *>(sm + L::SB + m0 / 64 * L::SBS + sw_off(tl, m0 % 64 / 8 + p)) = Vec16<__nv_bfloat16>::pack(v + 8 * p);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= decay;
                tmem_st16(at, v);
                tmem_st16(at + 16, v + 16);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kScaled]);
        }
    } else if (warp >= 8 && warp < 16) {
        const int half = (warp - 8) >> 2;
        for (int i = 0; i < nch; ++i) {
            const int c = i & 1;
            const StepArrays A(arrays + (i & 3) * SARR);
            ok = wait(kArr + (i & 3), (i >> 2) & 1) && wait(kG + c, (i >> 1) & 1);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // row tl, columns 64 half ..: blocks of 16 up to the one that row tl ends in, two at a time
            const uint32_t at = tm + lane_base + TG + 128 * c + 64 * half;
            const float ch = A.sh[tl], cl = A.sl[tl];
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int kb = 4 * half + k;
                uint32_t w[8];
                if (kb > 2 * q4 + 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                } else {
                    float v[16];
                    tmem_ld16(at + 16 * k, v);
                    tmem_wait_ld();
                    if (kb < 2 * q4) {  // wholly before my rows: one exponential for the block
                        const float f = ex2((ch - A.crefh[kb]) + (cl - A.crefl[kb]));
                        const ssm_f2 ff = ssm_pack(f, f);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(A.rs + 16 * kb + e);
                            const ssm_f2 lo = ssm_mul(ssm_pack(v[e], v[e + 1]), ssm_mul(ff, r.x));
                            const ssm_f2 hi = ssm_mul(ssm_pack(v[e + 2], v[e + 3]), ssm_mul(ff, r.y));
                            ssm_unpack(lo, v[e], v[e + 1]);
                            ssm_unpack(hi, v[e + 2], v[e + 3]);
                        }
                    } else if (A.span[kb] < 64.f) {
                        // as above, from the block's end: at most 2^64 too large before, and as much too small behind
                        const float f = ex2((ch - A.crefh[kb]) + (cl - A.crefl[kb]));
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int s = 16 * kb + e;
                            const float p = v[e] * (f * A.rs[s]);
                            v[e] = s <= tl ? p : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int s = 16 * kb + e;
                            const float p = v[e] * (ex2((ch - A.sh[s]) + (cl - A.sl[s])) * A.delta[s]);
                            v[e] = s <= tl ? p : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                }
                tmem_st8(at + 8 * k, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kP + c]);
        }
    } else if (warp >= 16) {
        const int jb = (warp - 16) >> 2 ? DP / 2 : 0;  // my half of the columns
        const float skip = a.D[h];
        const ssm_f2 skip2 = ssm_pack(skip, skip);
        for (int i = 0; i < nch; ++i) {
            const int c = i & 1;
            const uint32_t par = i & 1;
            const StepArrays A(arrays + (i & 3) * SARR);
            ok = wait(kArr + (i & 3), (i >> 2) & 1) && wait(kFullX + i % L::NX, (i / L::NX) & 1) && wait(kCX, par);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t at = tm + lane_base + TY;
            const float f = A.et[tl];
            const ssm_f2 ff = ssm_pack(f, f);
#pragma unroll 1
            for (int j = jb; j < jb + DP / 2; j += 32) {
                float v[32];
                tmem_ld16(at + j, v);
                tmem_ld16(at + j + 16, v + 16);
                tmem_wait_ld();
                const unsigned char *px = sm + L::X + i % L::NX * L::XB + j / 64 * SSLAB;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint4 xw = *reinterpret_cast<const uint4 *>(px + sw_off(tl, j % 64 / 8 + p));
                    const uint32_t x2[4] = {xw.x, xw.y, xw.z, xw.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float *o = v + 8 * p + 2 * k;
                        const ssm_f2 xf = ssm_pack(__uint_as_float(x2[k] << 16), __uint_as_float(x2[k] & 0xffff0000u));
                        ssm_unpack(ssm_fma(ff, ssm_pack(o[0], o[1]), ssm_mul(skip2, xf)), o[0], o[1]);
                    }
                }
                tmem_st16(at + j, v);
                tmem_st16(at + j + 16, v + 16);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kRows]);
            ok = wait(kY + c, (i >> 1) & 1);
            if (tid == 512) {
                mbar_arrive(&bar[kFreeArr + (i & 3)]);
                bulk_wait_read_all();  // the last output tile has left shared memory
            }
            if (named_any(2, 256, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            unsigned char *out = sm + L::OUT;
#pragma unroll 1
            for (int j = jb; j < jb + DP / 2; j += 32) {
                float v[32];
                tmem_ld16(at + j, v);
                tmem_ld16(at + j + 16, v + 16);
                tmem_wait_ld();
                if (j + 32 == jb + DP / 2) {  // the next chunk's c X_0 may go over Y
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[kFreeY]);
                }
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    *reinterpret_cast<uint4 *>(out + j / 64 * SSLAB + sw_off(tl, j % 64 / 8 + p)) = Vec16<__nv_bfloat16>::pack(v + 8 * p);
            }
            fence_proxy_async_smem();
            named_sync(2, 256);
            if (tid == 512) {
#pragma unroll
                for (int s = 0; s < DP / 64; ++s)
                    if (j0 + 64 * s < d) tma_store_4d(&tm_y, j0 + 64 * s, h, t_begin + i * SQ, b, out + s * SSLAB);
                bulk_commit();
                if (L::OUT_OVER_SB) {
                    bulk_wait_read_all();
                    mbar_arrive(&bar[kOut]);
                }
            }
        }
        if (tid == 512) bulk_wait_all();
    }
    if (!ok) *failed = 1;  // a wait ran out
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *failed) report_error(a.err, kErrWaitTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, TCOLS);
    }
}

// What the state kernel leaves: a part's last state (from state_in for the first part) and its
// log2 decay; or every chunk's by itself, or what every chunk passes on of its own adjoint (from dy
// and c in the places of x and b).
enum { kPart, kEach, kAdjoint };

// Parts are walked backwards.  The MMAs' sums are cut off, not rounded, so over a part's chunks the small
// bf16 parts of b have an accumulator of their own.  Chunks by themselves (of a.seg <= 128 positions each, `per` of a CTA)
// alternate between two accumulators, so that one is written out while the next is made.
template <int DP, int MP, int MODE>
__global__ void __launch_bounds__(STH, MP == 64 ? 2 : 1)
    ssm_state_kernel(ScanArgs a, int per, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b) {
    using L = SsmStateSmem<DP, MP>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);  // 0 copies, 1 MMAs
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 48);
    float *arrays = reinterpret_cast<float *>(sm + L::ARR);
    long long *tot = reinterpret_cast<long long *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int q4 = warp & 3, half = warp >> 2, tl = 32 * q4 + lane;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d;
    const int slices = (d + DP - 1) / DP, parts = a.segs * a.fine;
    constexpr bool EACH = MODE != kPart;
    // TMEM: the small parts have accumulators of their own (see above), so that parts that lie side by side
    // in shared memory are one MMA's columns (its A tile, x, is what an MMA's time goes to): all three
    // where they fit 256 columns, which leaves two CTAs an SM, else the high and the middle one
    constexpr int WIDE = MP == 64 && !EACH ? 3 : 2;  // parts of one MMA
    constexpr int ACC = WIDE * MP;                   // columns of an accumulator
    constexpr uint32_t COLS = EACH ? 2 * ACC : 256;
    const int groups = EACH ? (parts + per - 1) / per : a.state_segs;
    int id = blockIdx.x;
    const int seg = id % groups;
    id /= groups;
    const int j0 = id % slices * DP, unit = id / slices, b = unit / H, h = unit % H, g = h / (H / a.G);
    // positions of a chunk (the gradients' chunks have 64 where M > 64), and of the CTA
    constexpr int step = EACH && MP == 128 ? 64 : SQ;
    const int len = EACH ? step * per : a.seg / a.fine;
    const int t_begin = seg * len, t_end = min(N, t_begin + len);
    const int nch = t_end > t_begin ? (t_end - t_begin + step - 1) / step : 0;
    const __nv_bfloat16 *gdt = static_cast<const __nv_bfloat16 *>(a.dt) + (size_t)b * N * a.lddt + h;
    const float dt_bias = a.dt_bias[h];

    if ((s0 & 1023u) != 0u) {
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_b);
    }
    if (warp == 0) {
        tmem_alloc(tslot, COLS);
        tmem_relinquish();
    }
    const auto start_of = [&](int n) { return t_begin + (EACH ? n : nch - 1 - n) * step; };  // the n-th chunk walked
    const auto fetch = [&](int n) {  // one thread
        const int t0 = start_of(n);
        mbar_arrive_expect_tx(&bar[0], (uint32_t)(step * 128 * (DP / 64 + MP / 64)));
#pragma unroll
        for (int i = 0; i < MP / 64; ++i) tma_load_4d(sm + L::B + i * SSLAB, &tm_b, 64 * i, g, t0, b, &bar[0]);
#pragma unroll
        for (int i = 0; i < DP / 64; ++i) tma_load_4d(sm + L::X + i * SSLAB, &tm_x, j0 + 64 * i, h, t0, b, &bar[0]);
    };
    float dt_next = 0.f;
    const auto fetch_dt = [&](int n) {
        const int k = tid - SQ, p = start_of(n) + k;
        if (k >= 0) dt_next = n < nch && k < step && p < t_end ? __bfloat162float(gdt[(size_t)p * a.lddt]) : 0.f;
    };
    fetch_dt(0);
    Rate2 rate = {};
    if (tid >= SQ) rate = rate2_of(a.a_log[h]);
    __syncthreads();
    // the launches behind may take their places now: not before, a CTA of theirs that got this SM's TMEM
    // ahead of this one would wait for this one
    dependent_launch();
    if (tid == 0 && nch > 0) fetch(0);
    tc_fence_after();
    const uint32_t tm = *tslot;
    long long behind = 0;  // log2 a summed over the chunks done, in warps 4 .. 7
    const auto make_weights = [&](int n) {
        const int k = tid - SQ;
        if (k < 0) return;
        const bool in = k < step && start_of(n) + k < t_end;
        const float delta = in ? softplus(dt_next + dt_bias) : 0.f;
        long long all;
        const long long fx = chunk_sum(rate, delta, k, tot, all);
        if (MODE == kAdjoint)
            arrays[(n & 1) * SQ + k] = in ? ex2_fix(fx) : 0.f;
        else
            arrays[(n & 1) * SQ + k] = ex2_fix(all - fx + behind) * delta;
        if (!EACH) behind = max(behind + all, kFixLeast);
        if (MODE == kEach && k == 0 && j0 == 0) a.seg_log[(size_t)unit * parts + seg * per + n] = (float)all * kUnfix;
    };
    // the accumulator of chunk n (of the whole part) to memory
    const auto write_out = [&](int n, float *out, const float *in, float f) {
        // with DP = 64 lanes 64.. repeat 0..63 and take half of their columns
        constexpr int MH = DP == 64 ? MP / 4 : MP / 2;
        const int part = DP == 64 ? 2 * half + (q4 >> 1) : half, j = DP == 64 ? tl & 63 : tl;
#pragma unroll
        for (int blk = 0; blk < MH / 16; ++blk) {
            const int m0 = part * MH + 16 * blk;
            float v[16];
            const uint32_t at = tm + lane_base + (EACH && (n & 1) ? ACC : 0) + m0;
            tmem_ld16(at, v);
            float u[16], l[16];
            tmem_ld16(at + MP, u);
            if (WIDE > 2) tmem_ld16(at + 2 * MP, l);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += WIDE > 2 ? u[e] + l[e] : u[e];
            if (nch == 0)
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0.f;
            if (j0 + j < d)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (m0 + e < M) {
                        const size_t at = (size_t)(m0 + e) * d + j0 + j;
                        out[at] = in ? fmaf(f, __ldg(in + at), v[e]) : v[e];
                    }
        }
    };
    const auto each_out = [&](int n) { return a.seg_state + ((size_t)unit * parts + seg * per + n) * M * d; };
    if (nch > 0) make_weights(0);  // the last segment may have parts without a position
    fetch_dt(1);
    bool ok = true;
    int n = 0;
    for (; n < nch; ++n) {
        const uint32_t par = n & 1;
        ok = mbar_wait(&bar[0], par) && ok;
        if (__syncthreads_or(!ok)) break;  // the tiles and the weights are there
        // b times its weight: row r, half of the columns
        const int r = tid & 127, p0 = (tid >> 7) * (MP / 16);
        const float w = arrays[(n & 1) * SQ + r];
#pragma unroll
        for (int k = 0; k < MP / 16; ++k) {
            const int p = p0 + k;
            unsigned char *at = sm + L::B + p / 8 * SSLAB + sw_off(r, p % 8);
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
        tc_fence_before();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            // x^T as A: with DP = 64 its second 64 rows repeat the first
            const SmemDesc da = sw_desc(s0 + L::X, DP == 64 ? 0 : SSLAB);
            const SmemDesc dh = sw_desc(s0 + L::B, SSLAB);
            const SmemDesc dl = sw_desc(s0 + L::B + WIDE * (MP / 64) * SSLAB, SSLAB);
            const uint32_t acc = tm + (EACH && (n & 1) ? ACC : 0);
            constexpr uint32_t id_w = idesc(128, ACC, 1, 1, 1, 1), id_l = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll
            for (int k = 0; k < step / 16; ++k)
                mma_f16(acc, sw_step(da, k * 2048), sw_step(dh, k * 2048), id_w, (!EACH && n > 0) || k > 0);
            if (WIDE < PARTS)  // the low part joins the middle one
#pragma unroll
                for (int k = 0; k < step / 16; ++k)
                    mma_f16(acc + MP, sw_step(da, k * 2048), sw_step(dl, k * 2048), id_l, 1);
            mma_commit(&bar[1]);
        }
        __syncwarp();
        if (n + 1 < nch) {
            make_weights(n + 1);
            fetch_dt(n + 2);
        }
        if (EACH && n > 0) {  // the chunk before, whose MMAs have completed
            tc_fence_after();
            write_out(n - 1, each_out(n - 1), nullptr, 0.f);
        }
        if (n + 1 < nch) {
            ok = mbar_wait(&bar[1], par) && ok;
            if (tid == 0 && ok) fetch(n + 1);
        }
    }
    if (n == nch && nch > 0) ok = mbar_wait(&bar[1], (nch - 1) & 1) && ok;  // the last MMAs
    tc_fence_after();
    if (__syncthreads_or(!ok)) {  // a wait ran out
        if (tid == 0) {
            report_error(a.err, kErrWaitTimeout);
            if (n < nch) mbar_wait(&bar[0], n & 1);
        }
    } else if (EACH) {
        if (nch > 0) write_out(nch - 1, each_out(nch - 1), nullptr, 0.f);
    } else {
        // a single part's last state is the final state
        float *out = parts == 1 ? a.final_state + (size_t)unit * M * d : a.seg_state + ((size_t)unit * parts + seg) * M * d;
        if (tid == SQ) arrays[0] = (float)behind * kUnfix;
        __syncthreads();
        const float total = arrays[0];
        write_out(0, out, seg == 0 && a.state_in ? a.state_in + (size_t)unit * M * d : nullptr, ex2(total));
        if (tid == 0 && j0 == 0 && parts > 1) a.seg_log[(size_t)unit * parts + seg] = total;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, COLS);
    }
    // runs beside the launch before it, which it takes nothing from; what waits for this one waits for both
    if (MODE == kAdjoint) dependent_wait();
}

// Segment states, in place: seg_state[s] becomes the state before part s where a segment starts; the
// final state where it is wanted.  One thread per four state elements.
__global__ void __launch_bounds__(128) ssm_carry_kernel(ScanArgs a) {
    dependent_launch();
    dependent_wait();
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int n = a.M * a.d / 4, parts = a.segs * a.fine;
    const int unit = (int)(i / n), e = (int)(i % n);
    if (unit >= a.B * a.H) return;
    float4 *p = reinterpret_cast<float4 *>(a.seg_state + (size_t)unit * parts * a.M * a.d) + e;
    const float *lg = a.seg_log + (size_t)unit * parts;
    // the first part starts from the given state, which its last state holds
    float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in) X = __ldg(reinterpret_cast<const float4 *>(a.state_in + (size_t)unit * a.M * a.d) + e);
    constexpr int K = 8;
    for (int s0 = 0; s0 < parts; s0 += K) {
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
            if (s >= parts) break;
            if (s % a.fine == 0) p[(size_t)s * n] = X;  // a segment starts here
            if (s < a.state_segs) {
                const float w = ex2(f[k]);
                X = s == 0 ? v[k] : make_float4(fmaf(w, X.x, v[k].x), fmaf(w, X.y, v[k].y), fmaf(w, X.z, v[k].z), fmaf(w, X.w, v[k].w));
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

// Segments, and the parts of one whose states the first launch makes: the split with the least time
// by the launches' passes over the SMs, at 1.2 us a chunk in the chunk kernel (one CTA per SM) and 0.9 us
// in the state kernel (two), a CTA's start 3 us, the extra launches 5 us.  (Relative costs: a chunk takes
// longer where the launches fill the SMs.)  Measured against every other split, in us, without and with a
// final state, its choice first: 4 x 4096 positions of 16 heads of 128 x 64 58.6 and 72.6 in 2 segments of
// 4 parts, 63.2 and 82.0 of 8, 64.7 and 70.0 of 2, 73.3 and 76.0 in 4 segments, 64.6 and 138.6 in one;
// 1 x 14336 64.2 and 63.5 in 19 segments, 61.2 and 62.5 in 8 of 2 parts, 66.9 and 67.9 in 7; 1 x 8192 of 24
// heads of 64 x 128 72.8 and 73.2 in 6, 82.1 and 82.7 in 5; 2 x 4096 of 16 heads of 128 x 128 71.0 and 72.5
// in 4, 77.5 and 79.1 of 2 parts, 83.4 and 84.6 in 8.  Parts that fill the SMs several times over are not
// looked at: the search is short for long sequences too.
void ssm_chunk_segments(int B, int H, int N, int d, int M, int num_sms, int &seg, int &segs, int &fine) {
    const int nch = (N + SQ - 1) / SQ, dp = d <= 64 ? 64 : 128;
    const long long units = (long long)B * H * ((d + dp - 1) / dp), slots = (M <= 64 ? 2LL : 1LL) * num_sms;
    double best = 0;
    int pick = 1, pick_fine = 1;
    for (int s = 1; s <= nch && s <= 256; ++s) {
        const int per = (nch + s - 1) / s;
        if ((nch + per - 1) / per != s) continue;
        const double main = (double)((units * s + num_sms - 1) / num_sms) * (1.2 * per + 3.0);
        for (int f = 1; f <= (s > 1 ? per : 1); ++f) {
            if (f > 1 && units * (s - 1) * f > 4 * slots) break;
            if (per % f) continue;
            const double state = s > 1 ? (double)((units * (s - 1) * f + slots - 1) / slots) * (0.9 * (per / f) + 3.0) + 5.0 : 0.0;
            if ((s == 1 && f == 1) || main + state < best) {
                best = main + state;
                pick = s;
                pick_fine = f;
            }
        }
    }
    seg = (nch + pick - 1) / pick * SQ;
    segs = (N + seg - 1) / seg;
    fine = pick_fine;
}

template <int DP, int MP, int MODE>
static ida_status launch_states(const ScanArgs &a, cudaStream_t st) {
    constexpr int smem = SsmStateSmem<DP, MP>::TOTAL;
    static_assert(smem <= (MP == 64 ? 113 : 227) * 1024, "shared memory budget");
    CUtensorMap mx, mb;
    constexpr int step = MODE != kPart && MP == 128 ? 64 : SQ;
    ida_status s = ssm_map(&mx, a.x, a.B, a.N, a.H, a.d, a.ldx, step);
    if (s == IDA_OK) s = ssm_map(&mb, a.b, a.B, a.N, a.G, a.M, a.ldb, step);
    if (s != IDA_OK) return s;
    const auto kernel = ssm_state_kernel<DP, MP, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long units = (long long)a.B * a.H * ((a.d + DP - 1) / DP);
    // chunks by themselves: as many of a CTA as leave every SM its two (one where M > 64)
    const long long slots = MP == 64 ? 304 : 152, chunks = (long long)a.segs * a.fine;
    const int per = (int)((units * chunks + slots - 1) / slots < chunks ? (units * chunks + slots - 1) / slots : chunks);
    const long long groups = MODE == kPart ? a.state_segs : (chunks + per - 1) / per;
    if (MODE == kAdjoint) {
        e = launch_dependent(kernel, dim3((unsigned)(units * groups)), dim3(STH), smem, st, a, per, mx, mb);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, std::string("ssm adjoint states launch: ") + cudaGetErrorString(e));
    }
    kernel<<<(unsigned)(units * groups), STH, smem, st>>>(a, per, mx, mb);
    return launched("ssm segment states");
}

ida_status launch_ssm_states(const ScanArgs &a, cudaStream_t st) {
    if (a.d <= 64) return a.M <= 64 ? launch_states<64, 64, kPart>(a, st) : launch_states<64, 128, kPart>(a, st);
    return a.M <= 64 ? launch_states<128, 64, kPart>(a, st) : launch_states<128, 128, kPart>(a, st);
}

template <int DP, int MP>
static ida_status launch_each_of(const ScanArgs &a, bool rev, cudaStream_t st) {
    return rev ? launch_states<DP, MP, kAdjoint>(a, st) : launch_states<DP, MP, kEach>(a, st);
}
ida_status launch_ssm_chunk_states(const ScanArgs &a, bool rev, cudaStream_t st) {
    if (a.d <= 64) return a.M <= 64 ? launch_each_of<64, 64>(a, rev, st) : launch_each_of<64, 128>(a, rev, st);
    return a.M <= 64 ? launch_each_of<128, 64>(a, rev, st) : launch_each_of<128, 128>(a, rev, st);
}

template <int DP, int MP>
static ida_status launch_chunk(const ScanArgs &a, const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mc,
                               const CUtensorMap &my, cudaStream_t st) {
    constexpr int smem = SsmSmem<DP, MP>::TOTAL;
    static_assert(smem <= 227 * 1024, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(ssm_chunk_kernel<DP, MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long units = (long long)a.B * a.H * ((a.d + DP - 1) / DP);
    if (units * a.segs * a.fine > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows and heads");
    ida_status s = IDA_OK;
    if (a.state_segs > 0) s = launch_ssm_states(a, st);
    if (s != IDA_OK) return s;
    if (a.segs > 1) {
        const long long n = (long long)a.B * a.H * a.M * a.d / 4;
        e = launch_dependent(ssm_carry_kernel, dim3((unsigned)((n + 127) / 128)), dim3(128), 0, st, a);
        if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm segment sums launch: ") + cudaGetErrorString(e));
    }
    if (a.state_segs > 0)
        e = launch_dependent(ssm_chunk_kernel<DP, MP>, dim3((unsigned)(units * a.segs)), dim3(CTH), smem, st, a, mx, mb, mc, my);
    else
        ssm_chunk_kernel<DP, MP><<<(unsigned)(units * a.segs), CTH, smem, st>>>(a, mx, mb, mc, my);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm scan launch: ") + cudaGetErrorString(e));
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
