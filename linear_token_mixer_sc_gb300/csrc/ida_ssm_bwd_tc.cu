// ida_ssm_bwd_tc.cu -- the backward pass of the selective scan on the tcgen05 tensor cores (bf16
// inputs, d <= 128).
//
// Over a chunk of Q = 128 positions (64 where M > 64), with X_0 the state before it, Z the adjoint that reaches it
// from behind (a Z of the next position), S_t the running sum of log2 a, W_ts = 2^(S_t - S_s) for
// t >= s, f_s = 2^(S_Q - S_s), and the transposed products of positions
//   G [s][t] = b_s . c_t,   E [s][t] = x_s . dy_t          (MMAs, K = M and K = d)
// the gradients of ida_ssm_backward.cu's header are
//   dx_s = (D + D_s G_ss) dy_s + D_s (sum_{t > s} W G dy_t + f_s Z^T b_s)     P = D_s W G as A, dy as B
//   db_s = D_s (sum_t W E c_t + f_s Z x_s)                  R = D_s W E as A, c as B
//   dc_t = sum_s R b_s + 2^(S_t) X_0 dy_t                   R^T as A (the same tile read MN-major)
// and, from the fp32 K_st = D_s W G E (t > s, never rounded, never stored) and the inter-chunk
// products, the gradient of log a_t, the sum over all pairs (s < t <= u) of positions:
//   w_t = sum_{s < t <= u} K_su + sum_{u >= t} 2^(S_u) c_u^T X_0 dy_u + sum_{s < t} D_s f_s b_s^T Z x_s
//         + 2^(S_Q) <Z, X_0>.
// Its first sum is taken over groups of 16 positions, without differences but inside t's own group:
// there it is the running difference of K's row and column sums.  (One running difference over the
// whole chunk loses 3e-6 of a_log's gradient in heads that forget within a few positions.)  So dt's
// and the parameters' gradients come out to fp32 rounding although P and R are rounded to bf16 for
// the MMAs.  What enters w through MMAs is exact in its operands: b, c, x, dy are bf16, X_0 and Z are
// kept as the sum of three bf16 tiles.
//
// Chunks are independent: X_0 and Z of every chunk come from launch_ssm_chunk_states (forwards and
// backwards) and a running sum over the chunks.  One CTA of 512 threads takes the heads of one
// group (or a part of them) over one chunk: b, c and G once, db and dc added over the heads in TMEM,
// so that no per-head rows go to memory where a group's heads stay in one CTA.  Per head: E, then
// K, P and R on the CUDA cores (thread s of a lane quarter has row s; a warp sums K over its 32 rows
// by recursive halving), then the MMAs of dx, the inter-chunk products (read back, scaled by
// 2^S or f and added into db and dc) and the rest of db and dc.
//
// What bounds it: the stages of a head follow one another between block barriers (one CTA of 16 warps an
// SM: its registers and 175 KB are taken), at 0.34 instructions a cycle and scheduler; tensor pipe 12 %,
// HBM 15 %.  8 x 2048 positions of 12 heads of 64 x 64: 151 us, 98 of them this kernel's (8 us a head and
// chunk), 45 the chunk states' and 14 their running sums'.  (The MMAs issued by a 17th warp: 189 us, its
// threads' share of the registers spills the others'.)
//
// Waits are bounded as in ida_ssm_chunk.cu.
#include "ida_ssm_tc.cuh"

namespace ida {

using namespace tc;

constexpr int BTH = 512;  // threads per CTA

// Shared memory map; Q: positions, DP, MP: channels and state rows rounded up to 64 or 128.
template <int Q, int DP, int MP>
struct BwdSmem {
    static constexpr int SLAB = Q * 128;           // bytes of Q rows of 64 bf16
    static constexpr int XB = DP / 64 * SLAB, BB = MP / 64 * SLAB, QB = Q / 64 * SLAB;
    static constexpr int X = 0;                    // [DP / 64][Q s][64] bf16
    static constexpr int DY = X + XB;              // [DP / 64][Q t][64]
    static constexpr int B = DY + XB;              // [MP / 64][Q s][64]
    static constexpr int C = B + BB;               // [MP / 64][Q t][64]
    static constexpr int R = C + BB;               // [Q / 64][Q s][64 t]
    static constexpr int P = R + QB;               // [Q / 64][Q s][64 t], later dx [DP / 64][Q s][64]
    static constexpr int PSLAB = MP * 128, STS = 3 * PSLAB;  // a state's three parts [DP / 64][3][MP m][64]
    static constexpr int ST = P + (QB > XB ? QB : XB);  // parts of Z, later of X_0
    static constexpr int MISC = ST + DP / 64 * STS;
    static constexpr int ARR = MISC + 64;
    // S in two floats, 2^S, f, D and column factors of two heads; column sums of K in 8 parts and row
    // sums in 4 + 1, the inter-chunk products in 4 parts each, G and E of a position with itself
    static constexpr int NARR = 2 * 6 + 8 + 5 + 8 + 2;
    // <Z, X_0> per warp, 2^S_Q, parameters' parts; sums per warp; sums of K per pair of groups
    static constexpr int RED = ARR + NARR * SQ * 4;
    static constexpr int RATES = RED + 128 + 32 + 256;  // of 64 heads, made 32 at a time
    static constexpr int TOT = RATES + 512;
    static constexpr int TOTAL = TOT + 32;
};

// Columns.  With M <= 64 G stays for all heads and the inter-chunk products take E's place; with
// 64 positions and M > 64 they take G's and E's, and G is made again for every head.  Parts of a state
// side by side in shared memory are one MMA's columns, where there is room: all three, or the high and
// the middle one, which the low one then joins: 12 and 20 MMAs issued a head instead of 20 and 28.
template <int Q, int DP, int MP>
struct BwdTmem {
    static constexpr bool KEEP_G = MP == 64;
    static constexpr int WIDE = MP == 128 ? 1 : DP == 64 ? 3 : 2;  // parts of one MMA
    static constexpr uint32_t G = 0, E = KEEP_G ? 128 : 64, ZX = KEEP_G ? 128 : 0;
    static constexpr uint32_t DX = !KEEP_G ? 128 : DP == 64 ? 320 : 256, DB = KEEP_G ? 384 : 256, DC = KEEP_G ? 448 : 384, COLS = 512;
};

struct BwdTcArgs {
    ScanBwdArgs s;
    int splits;  // CTAs that share a group's heads; above 1, s.db_head and s.dc_head are [B][N][G][splits][M]
};

// three bf16 parts of 8 values
__device__ __forceinline__ void split3(const float *x, uint4 (&p)[3]) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[e];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        p[k] = Vec16<__nv_bfloat16>::pack(v);
        float h[8];
        Vec16<__nv_bfloat16>::unpack(p[k], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] -= h[e];
    }
}

template <int Q, int DP, int MP>
__global__ void __launch_bounds__(BTH, 1)
    ssm_bwd_tc_kernel(BwdTcArgs ba, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dy,
                      const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                      const __grid_constant__ CUtensorMap tm_dx) {
    using L = BwdSmem<Q, DP, MP>;
    using T = BwdTmem<Q, DP, MP>;
    constexpr int NG = Q / 16, MW = MP / 4;  // groups of 16 positions; state rows of a warp
    extern __shared__ __align__(1024) unsigned char sm[];
    const ScanBwdArgs &a = ba.s;
    const uint32_t s0 = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MISC);  // 0 b, c; 1 x, dy; 2 E and Z^T b; 3 dx, Z x; 4 the rest
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::MISC + 48);
    float *arr = reinterpret_cast<float *>(sm + L::ARR);
    float *ksum_t = arr + 12 * SQ;    // [8 groups of 16][128]: sum over the group's s of K, per t
    float *ksum_s = ksum_t + 8 * SQ;  // [4 warps of a quarter][128]: sum over their t of K / D_s, per s, ...
    float *kown = ksum_s + 4 * SQ;    // [128]: ... and over the t of s's own group
    float *zin = kown + SQ;           // [4][128]: b_s^T Z x_s
    float *xin = zin + 4 * SQ;      // [4][128]: c_t^T X_0 dy_t
    float *gs = xin + 4 * SQ, *es = gs + SQ;  // G and E at s = t
    float *red = reinterpret_cast<float *>(sm + L::RED);
    float *wsum = red + 32, *blk = wsum + 8;  // [8] and [8][8]
    Rate2 *rates = reinterpret_cast<Rate2 *>(sm + L::RATES);
    long long *tot = reinterpret_cast<long long *>(sm + L::TOT);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int q4 = warp & 3, wj = warp >> 2, row = 32 * q4 + lane;  // my lane of TMEM: position s or t
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int H = a.H, N = a.N, M = a.M, d = a.d, rep = H / a.G;
    int id = blockIdx.x;
    const int split = id % ba.splits;
    id /= ba.splits;
    const int g = id % a.G;
    id /= a.G;
    const int ch = id % a.chunks, b = id / a.chunks;
    const int t0 = ch * Q, len = min(Q, N - t0);
    const int per = (rep + ba.splits - 1) / ba.splits, r0 = split * per, r1 = min(rep, r0 + per);

    if ((s0 & 1023u) != 0u) {
        if (tid == 0) report_error(a.err, kErrShape);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_dy);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_c);
        tma_prefetch_desc(&tm_dx);
    }
    if (warp == 0) {
        tmem_alloc(tslot, T::COLS);
        tmem_relinquish();
    }
    const auto fetch = [&](int h) {  // one thread
        mbar_arrive_expect_tx(&bar[1], 2 * L::XB);
#pragma unroll
        for (int i = 0; i < DP / 64; ++i) {
            tma_load_4d(sm + L::X + i * L::SLAB, &tm_x, 64 * i, h, t0, b, &bar[1]);
            tma_load_4d(sm + L::DY + i * L::SLAB, &tm_dy, 64 * i, h, t0, b, &bar[1]);
        }
    };
    // one state [M][d]: read and split into its three parts, held in registers until their tiles
    // [m][j] may be written; with `other`, returns my share of <st, other>
    constexpr int NI = MP * DP / 8 / BTH;
    uint4 held[NI][3];
    const auto read_state = [&](const float *st, const float *other) {
        float dot = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = tid + n * BTH, m = i / (DP / 8), j = i % (DP / 8) * 8;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (m < M && j < d) {
                *reinterpret_cast<float4 *>(v) = __ldcg(reinterpret_cast<const float4 *>(st + (size_t)m * d + j));
                *reinterpret_cast<float4 *>(v + 4) = __ldcg(reinterpret_cast<const float4 *>(st + (size_t)m * d + j + 4));
                if (other) {
                    float u[8];
                    *reinterpret_cast<float4 *>(u) = __ldcg(reinterpret_cast<const float4 *>(other + (size_t)m * d + j));
                    *reinterpret_cast<float4 *>(u + 4) = __ldcg(reinterpret_cast<const float4 *>(other + (size_t)m * d + j + 4));
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot = fmaf(u[e], v[e], dot);
                }
            }
            split3(v, held[n]);
        }
        return dot;
    };
    const auto write_state = [&]() {
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = tid + n * BTH, m = i / (DP / 8), j = i % (DP / 8) * 8;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4 *>(sm + L::ST + j / 64 * L::STS + k * L::PSLAB + sw_off(m, j % 64 / 8)) = held[n][k];
        }
    };
    // step sizes and decays of head g rep + r, by warps 4 .. 7 (warp 0 issues MMAs), into the arrays of r's
    // parity
    const int ta = tid - SQ;
    float dt_next = 0.f;
    const auto read_dt = [&](int r) {
        if (ta >= 0 && ta < len && r < r1)
            dt_next = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.dt)[((size_t)b * N + t0 + ta) * a.lddt + g * rep + r]) + a.dt_bias[g * rep + r];
    };
    const auto make_arrays = [&](int r) {
        if (ta < 0 || ta >= SQ || r >= r1) return;
        if (((r - r0) & 31) == 0) {  // the rates of the next 32 heads
            if (warp == 4 && r + lane < r1) rates[((r - r0) & 63) + lane] = rate2_of(a.a_log[g * rep + r + lane]);
            named_sync(1, 128);
        }
        float *Sh = arr + ((r - r0) & 1) * 6 * SQ, *Sl = Sh + SQ, *et = Sl + SQ, *fs = et + SQ, *dl = fs + SQ, *rt = dl + SQ;
        const float delta = ta < len ? softplus(dt_next) : 0.f;
        long long all;
        const long long fx = chunk_sum(rates[(r - r0) & 63], delta, ta, tot, all);
        const float hi = (float)fx * kUnfix;
        // S at the end of the block of 16 before mine
        const int edge = (lane & 16) - 1;
        long long ref = __shfl_sync(0xffffffffu, fx, edge < 0 ? 0 : edge);
        if (edge < 0) ref = ta < 32 ? 0 : ta < 64 ? tot[0] : ta < 96 ? tot[0] + tot[1] : tot[0] + tot[1] + tot[2];
        Sh[ta] = hi;
        Sl[ta] = (float)(fx - (long long)(hi * kFix)) * kUnfix;
        et[ta] = ex2_fix(fx);
        fs[ta] = ex2_fix(all - fx);
        dl[ta] = delta;
        rt[ta] = ex2_fix(fx - ref);
        if (ta == 0) red[16 + 15 * ((r - r0) & 1)] = ex2_fix(all);
    };
    __syncthreads();
    dependent_launch();  // its TMEM is allocated
    dependent_wait();
    if (tid == 0 && r0 < r1) {
        mbar_arrive_expect_tx(&bar[0], 2 * L::BB);
#pragma unroll
        for (int i = 0; i < MP / 64; ++i) {
            tma_load_4d(sm + L::B + i * L::SLAB, &tm_b, 64 * i, g, t0, b, &bar[0]);
            tma_load_4d(sm + L::C + i * L::SLAB, &tm_c, 64 * i, g, t0, b, &bar[0]);
        }
        fetch(g * rep + r0);
    }
    tc_fence_after();
    const uint32_t tm = *tslot;
    // rows times the state's parts, K = d, by one thread
    const auto mma_state = [&](SmemDesc rows) {
        constexpr uint32_t id_w = idesc(128, T::WIDE * MP, 1, 1), id_m = idesc(128, MP, 1, 1);
#pragma unroll
        for (int part = T::WIDE > 1 ? 0 : 2; part >= 0; --part) {  // the small parts first: fewer roundings of the large sum
            const SmemDesc dz = sw_desc(s0 + L::ST + part * L::PSLAB, 16);
#pragma unroll 2
            for (int k = 0; k < DP / 16; ++k)
                mma_f16(tm + T::ZX, sw_step(rows, k / 4 * L::SLAB + k % 4 * 32), sw_step(dz, k / 4 * L::STS + k % 4 * 32), id_w,
                        (T::WIDE == 1 && part < 2) || k > 0);
        }
        if (T::WIDE == 2) {
            const SmemDesc dz = sw_desc(s0 + L::ST + 2 * L::PSLAB, 16);
#pragma unroll 2
            for (int k = 0; k < DP / 16; ++k)
                mma_f16(tm + T::ZX + MP, sw_step(rows, k / 4 * L::SLAB + k % 4 * 32), sw_step(dz, k / 4 * L::STS + k % 4 * 32), id_m, 1);
        }
    };
    // 16 columns of that product, with the tmem_ld16 that the caller has under way
    const auto read_zx = [&](int m, float (&v)[16]) {
        const uint32_t at = tm + lane_base + T::ZX + m;
        tmem_ld16(at, v);
        if (T::WIDE > 1) {
            float u[16], l[16];
            tmem_ld16(at + MP, u);
            if (T::WIDE > 2) tmem_ld16(at + 2 * MP, l);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += T::WIDE > 2 ? u[e] + l[e] : u[e];
        }
        tmem_wait_ld();
    };
    // 64 positions fill half the lanes: rows 64 .. 127 of the operands are whatever lies behind them in
    // shared memory, and the lanes that get them are not read
    const bool mine = row < Q;
    bool ok = true;
    read_dt(r0);
    make_arrays(r0);
    read_dt(r0 + 1);
    if (r0 < r1) read_state(a.adj + ((size_t)(b * H + g * rep + r0) * a.chunks + ch) * M * d, nullptr);
    // w, dt's gradient and the chunk's parts of the parameters', of the head before, by the warps that have
    // the fewest rows of K to make (the last quarter's).  Their sums are read before the next ones are
    // written, the rest runs beside the others' rows.
    struct Sums {
        float kc[NG], ks, zi, xi, ko, gg, ee, zx;
    };
    const auto read_sums = [&]() {
        const int t = 32 * wj + lane, J = t >> 4;
        Sums q = {};
        if (t < Q) {
#pragma unroll
            for (int k = 0; k < NG; ++k) q.kc[k] = k <= J ? ksum_t[k * SQ + t] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q.ks += ksum_s[k * SQ + t];
                q.zi += zin[k * SQ + t];
                q.xi += xin[k * SQ + t];
            }
            q.ko = kown[t];
            q.gg = gs[t];
            q.ee = es[t];
        }
#pragma unroll
        for (int k = 0; k < BTH / 32; ++k) q.zx += red[k];
        return q;
    };
    const auto finish = [&](int r, const Sums &q) {
        const int h = g * rep + r, unit = b * H + h;
        const uint32_t par = (r - r0) & 1;
        const float *et = arr + par * 6 * SQ + 2 * SQ, *fs = et + SQ, *dl = fs + SQ;
        const int t = 32 * wj + lane, J = t >> 4;
        float kc[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) kc[k] = q.kc[k];
        const float ks = q.ks, zi = q.zi, xi = q.xi, ko = q.ko, gg = q.gg, ee = q.ee, zx = q.zx;
        const float delta = t < Q ? dl[t] : 0.f, f = t < Q ? fs[t] : 0.f, e2 = t < Q ? et[t] : 0.f;
        const float rate = rates[(r - r0) & 63].hi * 0.6931471805599453f, zf = zi * f;
        float kt = 0.f, kd = 0.f;  // K of s in earlier groups, and in mine
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            kt += k < J ? kc[k] : 0.f;
            kd = k == J ? kc[k] : kd;
        }
        // over my group, from my position on: K from earlier groups, and inside the group the running
        // difference; before my position: K to later groups.  Over the warp: the inter-chunk terms
        float su = kt + (kd - delta * ko), sb = delta * ks, iu = e2 * xi, ib = delta * zf;
        const float own_b = sb, own_ib = ib;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, su, o), v = __shfl_up_sync(0xffffffffu, sb, o);
            const float x = __shfl_down_sync(0xffffffffu, iu, o), y = __shfl_up_sync(0xffffffffu, ib, o);
            if (o < 16) {
                if ((lane & 15) + o < 16) su += u;
                if ((lane & 15) >= o) sb += v;
            }
            if (lane + o < 32) iu += x;
            if (lane >= o) ib += y;
        }
        if (lane == 0) wsum[wj] = iu;
        if (lane == 31) wsum[4 + wj] = ib;
        // sums of K per pair of groups (s in group k, t in mine)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < NG; ++k) kc[k] += __shfl_xor_sync(0xffffffffu, kc[k], o);
        if ((lane & 15) == 0 && t < Q)
#pragma unroll
            for (int k = 0; k < NG; ++k) blk[k * 8 + J] = kc[k];
        named_sync(2, 128);
        float wt = su + (sb - own_b) + (iu + (ib - own_ib));
#pragma unroll
        for (int k = 0; k < 4; ++k) wt += k > wj ? wsum[k] : k < wj ? wsum[4 + k] : 0.f;
#pragma unroll
        for (int i = 0; i < NG - 2; ++i)  // pairs of groups around mine
#pragma unroll
            for (int k = i + 2; k < NG; ++k) wt += i < J && k > J ? blk[i * 8 + k] : 0.f;
        wt = fmaf(zx, red[16 + 15 * par], wt);
        float ga = 0.f, gb = 0.f, gd = 0.f;
        if (t < len) {
            // 1 / (1 + e^-z) of D = log(1 + e^z) is 1 - e^-D
            const float ddt = (ks + ko + gg * ee + zf - rate * wt) * -expm1f(-delta);
            static_cast<__nv_bfloat16 *>(a.ddt)[((size_t)b * N + t0 + t) * a.ldddt + h] = __float2bfloat16_rn(ddt);
            ga = -rate * (delta * wt);  // 0 where wt is, whatever the rate
            gb = ddt;
            gd = ee;
        }
        ga = warp_sum(ga);
        gb = warp_sum(gb);
        gd = warp_sum(gd);
        if (lane == 0)
            *reinterpret_cast<float4 *>(a.part + (((size_t)unit * a.chunks + ch) * 4 + wj) * 4) = make_float4(ga, gb, gd, 0.f);
    };
    int r = r0;
    for (; r < r1; ++r) {
        const int h = g * rep + r, unit = b * H + h;
        const uint32_t par = (r - r0) & 1;
        const size_t so = ((size_t)unit * a.chunks + ch) * M * d;
        const float *Sh = arr + par * 6 * SQ, *Sl = Sh + SQ, *et = Sl + SQ, *fs = et + SQ, *dl = fs + SQ, *rt = dl + SQ;
        write_state();  // Z
        fence_proxy_async_smem();
        if (r == r0) ok = mbar_wait(&bar[0], 0) && ok;
        ok = mbar_wait(&bar[1], par) && ok;
        if (__syncthreads_or(!ok)) break;
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const SmemDesc dxk = sw_desc(s0 + L::X, 16), dyk = sw_desc(s0 + L::DY, 16);
            const SmemDesc db = sw_desc(s0 + L::B, 16), dc = sw_desc(s0 + L::C, 16), dz = sw_desc(s0 + L::ST, L::STS);
            constexpr uint32_t id_q = idesc(128, Q, 1, 1), id_x = idesc(128, DP, 1, 1, 0, 1);
#pragma unroll 2
            for (int k = 0; k < DP / 16; ++k)
                mma_f16(tm + T::E, sw_step(dxk, k / 4 * L::SLAB + k % 4 * 32), sw_step(dyk, k / 4 * L::SLAB + k % 4 * 32), id_q, k > 0);
            if (r == r0 || !T::KEEP_G)
#pragma unroll 2
                for (int k = 0; k < MP / 16; ++k)
                    mma_f16(tm + T::G, sw_step(db, k / 4 * L::SLAB + k % 4 * 32), sw_step(dc, k / 4 * L::SLAB + k % 4 * 32), id_q, k > 0);
            // Z^T b: Z's high part [K = m][j] as an MN-major B
#pragma unroll 2
            for (int k = 0; k < MP / 16; ++k)
                mma_f16(tm + T::DX, sw_step(db, k / 4 * L::SLAB + k % 4 * 32), sw_step(dz, k * 2048), id_x, k > 0);
            mma_commit(&bar[2]);
        }
        __syncwarp();
        if (tid == 0) bulk_wait_read_all();  // dx of the last head has left P's place
        Sums last = {};
        if (r > r0 && q4 == 3) last = read_sums();
        ok = mbar_wait(&bar[2], par);
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (mine) {  // Z^T b D_s f_s: my row, a quarter of the channels
            const float f = dl[row] * fs[row];
            constexpr int CW = DP / 4;
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
                float v[16];
                tmem_ld16(tm + lane_base + T::DX + wj * CW + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= f;
                tmem_st16(tm + lane_base + T::DX + wj * CW + c, v);
            }
        }
        if (r > r0 && q4 == 3) finish(r - 1, last);
        if (mine) {
            // K, P, R: row s, every fourth block of 16 columns t
            const float sh = Sh[row], sl = Sl[row], delta = dl[row];
            float ks = 0.f;
#pragma unroll 1
            for (int i = 0; i < NG / 4; ++i) {
                const int kb = wj + 4 * i;
                uint4 pp[2], rr[2];
                if (kb < 2 * q4) {  // wholly before my rows
#pragma unroll
                    for (int e = 0; e < 2; ++e) pp[e] = rr[e] = make_uint4(0, 0, 0, 0);
                    ksum_t[(2 * q4 + (lane >> 4)) * SQ + 16 * kb + (lane & 15)] = 0.f;
                } else {
                    float gv[16], ev[16], kk[16];
                    tmem_ld16(tm + lane_base + T::G + 16 * kb, gv);
                    tmem_ld16(tm + lane_base + T::E + 16 * kb, ev);
                    tmem_wait_ld();
                    if (kb >= 2 * q4 + 2) {  // wholly behind my rows: decay to the block's start, then inside it
                        const float f = ex2((Sh[16 * kb - 1] - sh) + (Sl[16 * kb - 1] - sl));
                        const ssm_f2 ff = ssm_pack(f, f), dd = ssm_pack(delta, delta);
                        ssm_f2 sum = 0ull;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const ssm_f2 w = ssm_mul(ff, *reinterpret_cast<const ssm_f2 *>(rt + 16 * kb + e));
                            const ssm_f2 gg = ssm_pack(gv[e], gv[e + 1]), we = ssm_mul(w, ssm_pack(ev[e], ev[e + 1]));
                            const ssm_f2 k1 = ssm_mul(we, gg), one = ssm_pack(1.f, 1.f);
                            sum = ssm_fma(k1, one, sum);
                            ssm_unpack(ssm_mul(k1, dd), kk[e], kk[e + 1]);
                            ssm_unpack(ssm_mul(gg, ssm_mul(w, dd)), gv[e], gv[e + 1]);
                            ssm_unpack(ssm_mul(we, dd), ev[e], ev[e + 1]);
                        }
                        float lo, hi;
                        ssm_unpack(sum, lo, hi);
                        ks += lo + hi;
                    } else {
                        // selects, no branches: a warp's rows take different ones (K, P and R of a head took 5400
                        // cycles with them, 4600 without)
                        float ko = 0.f, go = 0.f, eo = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int t = 16 * kb + e;
                            const float diff = (Sh[t] - sh) + (Sl[t] - sl);
                            const float w = ex2(t > row ? diff : -INFINITY), k0 = w * ev[e] * gv[e];
                            const float k1 = t > row ? k0 : 0.f;
                            ko += k1;
                            kk[e] = k1 * delta;
                            go = t == row ? gv[e] : go;
                            eo = t == row ? ev[e] : eo;
                            const float p = gv[e] * (w * delta), q = ev[e] * ((t == row ? 1.f : w) * delta);
                            gv[e] = t > row ? p : 0.f;
                            ev[e] = t >= row ? q : 0.f;
                        }
                        if (kb == row >> 4) {
                            kown[row] = ko;
                            gs[row] = go;
                            es[row] = eo;
                        } else {
                            ks += ko;
                        }
                    }
                    pp[0] = Vec16<__nv_bfloat16>::pack(gv);
                    pp[1] = Vec16<__nv_bfloat16>::pack(gv + 8);
                    rr[0] = Vec16<__nv_bfloat16>::pack(ev);
                    rr[1] = Vec16<__nv_bfloat16>::pack(ev + 8);
                    // summed over my half warp's rows: lane l ends with column l % 16 of the block
#pragma unroll
                    for (int n = 8; n >= 1; n >>= 1) {
                        const bool up = (lane & n) != 0;
#pragma unroll
                        for (int k = 0; k < n; ++k) {
                            const float send = up ? kk[k] : kk[k + n], keep = up ? kk[k + n] : kk[k];
                            kk[k] = keep + __shfl_xor_sync(0xffffffffu, send, n);
                        }
                    }
                    ksum_t[(2 * q4 + (lane >> 4)) * SQ + 16 * kb + (lane & 15)] = kk[0];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int off = kb / 4 * L::SLAB + sw_off(row, kb % 4 * 2 + e);
                    *reinterpret_cast<uint4 *>(sm + L::P + off) = pp[e];
                    *reinterpret_cast<uint4 *>(sm + L::R + off) = rr[e];
                }
            }
            ksum_s[wj * SQ + row] = ks;
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const SmemDesc dp = sw_desc(s0 + L::P, 16), dyn = sw_desc(s0 + L::DY, L::SLAB), dxk = sw_desc(s0 + L::X, 16);
            constexpr uint32_t id_x = idesc(128, DP, 1, 1, 0, 1), id_c = idesc(128, MP, 1, 1, 1, 1);
#pragma unroll 2
            for (int k = 0; k < Q / 16; ++k)
                mma_f16(tm + T::DX, sw_step(dp, k / 4 * L::SLAB + k % 4 * 32), sw_step(dyn, k * 2048), id_x, 1);
            mma_state(dxk);
            mma_commit(&bar[3]);
            // R^T b into dc, beside what is done with the products before it
            const SmemDesc drt = sw_desc(s0 + L::R, Q == 64 ? 0 : L::SLAB);  // 64 positions: rows 64.. repeat them
            const SmemDesc dbn = sw_desc(s0 + L::B, L::SLAB);
#pragma unroll 2
            for (int k = 0; k < Q / 16; ++k)
                mma_f16(tm + T::DC, sw_step(drt, k * 2048), sw_step(dbn, k * 2048), id_c, r > r0 || k > 0);
        }
        __syncwarp();
        const float cross = warp_sum(read_state(a.state0 + so, a.adj + so));
        ok = mbar_wait(&bar[3], par);
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (lane == 0) red[warp] = cross;
        write_state();  // X_0's parts take the place of Z's
        if (mine) {  // dx out: my row, a quarter of the channels, over P; its own dy's term in fp32
            constexpr int CW = DP / 4;
            const float own = fmaf(dl[row], gs[row], a.D[h]);
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
                const int j = wj * CW + c;
                float v[16], u[16];
                tmem_ld16(tm + lane_base + T::DX + j, v);
                const unsigned char *py = sm + L::DY + j / 64 * L::SLAB;
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(py + sw_off(row, j % 64 / 8)), u);
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(py + sw_off(row, j % 64 / 8 + 1)), u + 8);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = fmaf(own, u[e], v[e]);
                unsigned char *out = sm + L::P + j / 64 * L::SLAB;
                *reinterpret_cast<uint4 *>(out + sw_off(row, j % 64 / 8)) = Vec16<__nv_bfloat16>::pack(v);
                *reinterpret_cast<uint4 *>(out + sw_off(row, j % 64 / 8 + 1)) = Vec16<__nv_bfloat16>::pack(v + 8);
            }
        }
        if (mine) {  // Z x: its product with b, and D_s f_s of it into db
            const float f = dl[row] * fs[row];
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < MW; c += 16) {
                const int m = MW * wj + c;
                float v[16], u[16], w[16];
                if (r > r0) tmem_ld16(tm + lane_base + T::DB + m, w);
                read_zx(m, v);
                const unsigned char *pb = sm + L::B + m / 64 * L::SLAB;
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(pb + sw_off(row, m % 64 / 8)), u);
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(pb + sw_off(row, m % 64 / 8 + 1)), u + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    dot = fmaf(u[e], v[e], dot);
                    v[e] = r > r0 ? fmaf(f, v[e], w[e]) : f * v[e];
                }
                tmem_st16(tm + lane_base + T::DB + m, v);
            }
            zin[wj * SQ + row] = dot;
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const SmemDesc dyk = sw_desc(s0 + L::DY, 16), dr = sw_desc(s0 + L::R, 16);
            const SmemDesc dcn = sw_desc(s0 + L::C, L::SLAB);
            constexpr uint32_t id_b = idesc(128, MP, 1, 1, 0, 1);
            mma_state(dyk);
#pragma unroll 2
            for (int k = 0; k < Q / 16; ++k)
                mma_f16(tm + T::DB, sw_step(dr, k / 4 * L::SLAB + k % 4 * 32), sw_step(dcn, k * 2048), id_b, 1);
            mma_commit(&bar[4]);
        }
        __syncwarp();
        if (tid == 0) {
#pragma unroll
            for (int s = 0; s < DP / 64; ++s)
                if (64 * s < d) tma_store_4d(&tm_dx, 64 * s, h, t0, b, sm + L::P + s * L::SLAB);
            bulk_commit();
        }
        if (r + 1 < r1) {  // the next head's arrays and Z
            make_arrays(r + 1);
            read_dt(r + 2);
            read_state(a.adj + so + (size_t)a.chunks * M * d, nullptr);
        }
        ok = mbar_wait(&bar[4], par);
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (tid == 0 && r + 1 < r1) fetch(h + 1);
        if (mine) {  // X_0 dy: its product with c, and 2^S_t of it into dc
            const float f = et[row];
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < MW; c += 16) {
                const int m = MW * wj + c;
                float v[16], u[16], w[16];
                tmem_ld16(tm + lane_base + T::DC + m, w);
                read_zx(m, v);
                const unsigned char *pc = sm + L::C + m / 64 * L::SLAB;
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(pc + sw_off(row, m % 64 / 8)), u);
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(pc + sw_off(row, m % 64 / 8 + 1)), u + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    dot = fmaf(u[e], v[e], dot);
                    v[e] = fmaf(f, v[e], w[e]);
                }
                tmem_st16(tm + lane_base + T::DC + m, v);
            }
            xin[wj * SQ + row] = dot;
        }
        tmem_wait_st();
        tc_fence_before();
    }
    if (r == r1 && r > r0) {
        __syncthreads();
        if (q4 == 3) finish(r - 1, read_sums());
    }
    if (r < r1) {  // a wait ran out
        if (tid == 0) {
            report_error(a.err, kErrWaitTimeout);
            mbar_wait(&bar[0], 0);
            mbar_wait(&bar[1], (r - r0) & 1);
        }
    } else {
        // db and dc of the group (or of this CTA's heads): my row, a quarter of the state rows
        if (mine)
#pragma unroll
            for (int k = 0; k < 2 * MW / 16; ++k) {
                const bool is_c = k >= MW / 16;
                const int m0 = MW * wj + k % (MW / 16) * 16;
                float v[16];
                tmem_ld16(tm + lane_base + (is_c ? T::DC : T::DB) + m0, v);
                tmem_wait_ld();
                if (row < len) {
                    const size_t at = (size_t)b * N + t0 + row;
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        const int m = m0 + e;
                        if (m >= M) break;
                        if (ba.splits == 1) {
                            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(is_c ? a.dc : a.db) + at * (is_c ? a.lddc : a.lddb) + g * M + m;
                            *reinterpret_cast<uint4 *>(o) = Vec16<__nv_bfloat16>::pack(v + e);
                        } else {
                            float4 *o = reinterpret_cast<float4 *>((is_c ? a.dc_head : a.db_head) + ((at * a.G + g) * ba.splits + split) * M + m);
                            o[0] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                            o[1] = make_float4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
                        }
                    }
                }
            }
    }
    if (tid == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, T::COLS);
    }
}

// ---- host side ---------------------------------------------------------------------------

// CTAs that share a group's heads: the fewest passes over the SMs, a head and chunk taking about 7.5 us
// and a CTA's start 6 more; the partial rows of a shared group cost their traffic at about 5 TB/s.
int ssm_bwd_tc_chunk(int M) { return M <= 64 ? 128 : 64; }
int ssm_bwd_tc_splits(int B, int H, int N, int G, int M) {
    const int rep = H / G, q = ssm_bwd_tc_chunk(M);
    const long long base = (long long)B * ((N + q - 1) / q) * G;
    int best = 1;
    double cost = 0;
    for (int s = 1; s <= rep; ++s) {
        const int per = (rep + s - 1) / s;
        if ((rep + per - 1) / per != s) continue;  // some CTA would have no head
        const double c = (double)((base * s + 151) / 152) * (7.5 * per + 6.0) +
                         (s > 1 ? 5.0 + 16.0 * (double)B * N * G * s * M / 5e6 : 0.0);
        if (s == 1 || c < cost) {
            best = s;
            cost = c;
        }
    }
    return best;
}

template <int Q, int DP, int MP>
static ida_status launch_bwd_tc_d(const BwdTcArgs &ba, cudaStream_t st) {
    const ScanBwdArgs &a = ba.s;
    constexpr int smem = BwdSmem<Q, DP, MP>::TOTAL;
    static_assert(smem <= 227 * 1024, "shared memory budget");
    CUtensorMap mx, mdy, mb, mc, mdx;
    ida_status s = ssm_map(&mx, a.x, a.B, a.N, a.H, a.d, a.ldx, Q);
    if (s == IDA_OK) s = ssm_map(&mdy, a.dy, a.B, a.N, a.H, a.d, (long long)a.H * a.d, Q);
    if (s == IDA_OK) s = ssm_map(&mb, a.b, a.B, a.N, a.G, a.M, a.ldb, Q);
    if (s == IDA_OK) s = ssm_map(&mc, a.c, a.B, a.N, a.G, a.M, a.ldc, Q);
    if (s == IDA_OK) s = ssm_map(&mdx, a.dx, a.B, a.N, a.H, a.d, a.lddx, Q);
    if (s != IDA_OK) return s;
    cudaError_t e = cudaFuncSetAttribute(ssm_bwd_tc_kernel<Q, DP, MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long ctas = (long long)a.B * a.chunks * a.G * ba.splits;
    if (ctas > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many positions and groups");
    e = launch_dependent(ssm_bwd_tc_kernel<Q, DP, MP>, dim3((unsigned)ctas), dim3(BTH), smem, st, ba, mx, mdy, mb, mc, mdx);
    return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, std::string("ssm scan backward launch: ") + cudaGetErrorString(e));
}

// The chunk states, forwards and backwards, from zero.
ida_status launch_bwd_tc_states(const ScanBwdArgs &a, cudaStream_t st) {
    ScanArgs f = {a.x, a.b, a.c, a.dt, a.a_log, a.dt_bias, a.D, nullptr, nullptr, nullptr, a.B, a.H, a.N, a.d, a.G, a.M,
                  a.ldx, a.ldb, a.ldc, a.lddt, a.chunk, a.chunks, 1, a.chunks, a.state0, a.chunk_log, a.err};
    ida_status s = launch_ssm_chunk_states(f, false, st);
    if (s != IDA_OK) return s;
    f.x = a.dy;
    f.b = a.c;
    f.ldx = (long long)a.H * a.d;
    f.ldb = a.ldc;
    f.seg_state = a.adj;
    return launch_ssm_chunk_states(f, true, st);
}

ida_status launch_bwd_tc(const ScanBwdArgs &a, int splits, cudaStream_t st) {
    const BwdTcArgs ba = {a, splits};
    if (a.M <= 64) return a.d <= 64 ? launch_bwd_tc_d<128, 64, 64>(ba, st) : launch_bwd_tc_d<128, 128, 64>(ba, st);
    return a.d <= 64 ? launch_bwd_tc_d<64, 64, 128>(ba, st) : launch_bwd_tc_d<64, 128, 128>(ba, st);
}

}  // namespace ida
