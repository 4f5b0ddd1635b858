// ida_gemm.cuh -- matrix products of the feed-forward block on the tensor cores: one persistent
// kernel over pairs of SMs, with the epilogues that fuse what follows a product.
//
// A pair of CTAs (a cluster of two, tcgen05 cta_group::2) owns an output tile of 256 rows x 256
// columns: each CTA brings its 128 rows of A and half of the 256 columns of B into shared memory by
// TMA, the even one issues the MMAs for both, and each finds its own 128 rows x 256 columns in its
// TMEM, where two such accumulators fit, so that one tile's epilogue runs beside the next one's MMAs.
// A pair tile reads 64 KB for 8.4 MFLOP; with one CTA a tile of 128 x 256 would read 48 KB for half of
// that, 96 bytes a clock of every SM at the MMA's rate, more than the L2 gives.
//
// Warps: 0 loads, 1 issues the MMAs (of the even CTA), the others are the epilogue's.  The direct kind
// accumulates a whole tile in TMEM.  The others take the accumulator out every `chunk` contraction
// blocks and add it up in registers, scaled in e4m3, where each block of 128 has scales of its own: the
// tensor cores cut a running sum off, by up to 2^-23 of it every 16 elements and always towards zero, which
// fp32 inputs (three bf16 parts, six products) show after 512 elements and bf16 results after many rows (weights'
// gradients of one sign over 2^20 rows came out 1.6e-3 too small).
#pragma once

#include <cuda.h>
#include <cuda_fp8.h>

#include "ida_vec.cuh"
#include "tc_sm103.cuh"

namespace ida {

enum { kDirect = 0, kSums = 1, kE4M3 = 2 };           // bf16 (or parts) summed in TMEM, or in registers by chunks; e4m3
enum { kPlain = 0, kGate = 1, kGateBwd = 2 };         // epilogues
constexpr int GOP = 128 * 128;                        // bytes of an operand of a stage
constexpr int GSLAB = 32 * 128;                       // bytes of a warp's staged box: 32 rows of 128 bytes
// Warps of the epilogue.  The gate's and its gradients' have work for eight (gradients of 16384 rows of 768 and 2048
// channels 61 us with four, 55 with eight).  Sums in registers are eight warps', 128 a thread (14336 rows' gated
// projection in 8 bits 247 us; 280 with sixteen warps and 64, 307 with those and halves of the accumulator released by
// themselves: an MMA of half the columns reads A again, and shared memory cannot feed that).
constexpr int GEW = 8;
constexpr int gemm_threads(int kind) { return (kind == kDirect ? 64 : 128) + 32 * GEW; }
// Boxes that a warp stages, and the stages that shared memory has left for operands
constexpr int gemm_boxes(int epi) { return epi == kGateBwd ? 2 : 1; }
constexpr int gemm_staging(int epi) { return GEW * gemm_boxes(epi) * GSLAB; }
constexpr int gemm_stages(int epi) {
    const int n = (227 * 1024 - 1024 - 512 - gemm_staging(epi)) / (2 * GOP);
    return n < 6 ? n : 6;
}
constexpr int gemm_smem(int epi) { return gemm_stages(epi) * 2 * GOP + gemm_staging(epi) + 1024 + 512; }
constexpr int GST = 6;                                // stages at most

struct GemmSeg {
    unsigned char a, ap, b, bp;  // maps and parts of one pass over the contraction
};

// n / d for n < 2^31 without a division (every warp places its own tiles, and divisions took 1100 .. 1700
// clocks a tile, a tenth of a tile's time in 8 bits): with 2^s >= d and m = 2^32 (2^s - d) / d + 1 rounded
// down,  n / d = (m n / 2^32 + n) / 2^s.
struct Divisor {
    unsigned m, s, d;
};
inline Divisor divisor(unsigned d) {
    unsigned s = 0;
    while ((1ull << s) < d) ++s;
    return {(unsigned)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, d};
}
__device__ __forceinline__ int divide(int n, const Divisor &d) { return (int)((__umulhi(d.m, (unsigned)n) + (unsigned)n) >> d.s); }

struct GemmArgs {
    CUtensorMap a[3], b[3], o[2], e[2];  // operands; boxes that the epilogue writes and reads
    int M[3], N[3];                      // rows and columns of each problem's output
    int tiles, bands[3], count[3];       // of the launch; whole bands of 8 rows of tiles, and tiles, of each problem
    Divisor band[3], last[3];            // tiles of such a band, rows of tiles of the last one (1 if there is none)
    void *out[3];                        // outputs: of each problem; kGate: the product and its factors
    int split;                           // pairs that share a tile's contraction
    int back;                            // tiles from the last to the first: the rows that the launch before wrote
                                         // last are in the L2 (block of 16384 rows of 2048 channels 569 us, then 563)
    int problems, segs, kblocks, chunk;  // kblocks: blocks of 128 bytes along each segment's contraction
    GemmSeg seg[12];
    int keep;                            // kGate: store the two factors as well
    const float *sa, *sb[2];             // kE4M3: scales [M, kblocks] and [ceil(N / 128), kblocks] (one or two of b)
    float *so;                           // kE4M3 kGate: output scales [M, ceil(N / 128)]
    unsigned *err;
};

// ---- what only pairs need ------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of a shared variable of the cluster's CTA `rank`; of the pair's even one
__device__ __forceinline__ uint32_t cluster_addr(const void *p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t lead_addr(const void *p) { return cluster_addr(p, (int)cluster_rank() & ~1); }
__device__ __forceinline__ float4 cluster_float4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// No data but the accumulator's goes with this arrival, and tcgen05's own fence orders that: a release at the
// cluster's scope would wait for all of the warp's memory accesses (14336 rows' gated projection in 8 bits
// 649 us with it, 330 without).
__device__ __forceinline__ void arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void arrive_local(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// Waits of about two seconds at most; the role that gives up reports it and ends, and the others follow.
__device__ __forceinline__ bool pair_wait(uint64_t *bar, uint32_t parity, unsigned *err) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity))
        if (clock64() - t0 > 4000000000LL) {
            report_error(err, kErrWaitTimeout);
            return false;
        }
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned *err) {  // by a whole warp
    return __all_sync(0xffffffffu, pair_wait(bar, parity, err));
}
__device__ __forceinline__ void pair_load(void *dst, const void *map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_3d(void *dst, const void *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void store_3d(const void *map, int c0, int c1, int c2, const void *src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(src))
                 : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t *bar) {  // to both CTAs' copies of the barrier
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_u32(bar)),
        "h"((unsigned short)(3 << (cluster_rank() & ~1)))
        : "memory");
}
template <bool E4M3>
__device__ __forceinline__ void pair_mma(uint32_t d, tc::SmemDesc a, tc::SmemDesc b, uint32_t id, uint32_t acc) {
    if (E4M3)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
            "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
            "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(id), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
            "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
            "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(id), "r"(acc)
            : "memory");
}
// 32 lanes x 32 columns; the values are there after tc::tmem_wait_ld()
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_use(uint32_t (&r)[N]) {  // keeps uses of r behind the wait
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// (x0, x1) += (v0, v1) m, two at a time
__device__ __forceinline__ void add_scaled(float &x0, float &x1, uint32_t v0, uint32_t v1, float m) {
    asm("{\n\t.reg .b64 x, v, m;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\t"
        "fma.rn.f32x2 x, v, m, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "r"(v0), "r"(v1), "f"(m));
}

// Shared-memory descriptor of a 128-byte-swizzled operand (rows of 128 bytes, 1024 bytes between groups of
// 8; `lbo` between 64-element slabs of MN-major operands) and the byte offset of 16-byte piece c of row r.
__device__ __forceinline__ tc::SmemDesc pair_desc(uint32_t addr, uint32_t lbo) {
    return {((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16), (1024u >> 4) | (1u << 14) | (2u << 29)};
}
__device__ __forceinline__ int swz128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// ---- the activation --------------------------------------------------------------------------

// 1 / (1 + e^-x): for bf16 results from the hardware's exponential and reciprocal themselves (off by (|x| + 8) 2^-24
// of its size; what lies below 2^-126 is 0; by __expf and __fdividef 14336 rows' gated projection in 8 bits takes 3 us
// more), else by expf and a division
constexpr float kLog2E = 1.4426950408889634f, kLog2ERest = 1.9259630e-8f;
template <typename E>
__device__ __forceinline__ float sigmoid(float x) {
    if constexpr (sizeof(E) == 4) return 1.f / (1.f + expf(-x));
    float e, r;
    // log2 e in two floats: by one alone the exponential is off by another 0.22 |x| 2^-24 (the time is the same)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(x, -kLog2E, x * -kLog2ERest)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// silu(x0) u0 and silu(x1) u1 for 8-bit results, over x0 and x1: the same operations, two at a time but for the
// hardware's own (14336 rows' gated projection 251 us one by one, so 249)
__device__ __forceinline__ void gate_two(float &x0, float &x1, float u0, float u1) {
    asm("{\n\t.reg .b64 x, u, h, l, n, t;\n\t.reg .f32 a, b;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 u, {%2, %3};\n\t"
        "mov.b64 h, {%4, %4};\n\tmov.b64 l, {%5, %5};\n\tmov.b64 n, {%6, %6};\n\t"
        "mul.rn.f32x2 t, x, l;\n\tfma.rn.f32x2 t, x, h, t;\n\tmov.b64 {a, b}, t;\n\t"
        "ex2.approx.ftz.f32 a, a;\n\tex2.approx.ftz.f32 b, b;\n\tmov.b64 t, {a, b};\n\t"
        "add.rn.f32x2 t, t, n;\n\tmov.b64 {a, b}, t;\n\t"
        "rcp.approx.ftz.f32 a, a;\n\trcp.approx.ftz.f32 b, b;\n\tmov.b64 t, {a, b};\n\t"
        "mul.rn.f32x2 x, x, t;\n\tmul.rn.f32x2 x, x, u;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(u0), "f"(u1), "f"(-kLog2E), "f"(-kLog2ERest), "f"(1.f));
}

// ---- tiles -----------------------------------------------------------------------------------

struct GemmTile {
    int p, row0, col0;  // problem, the pair's first row and column (kGate: of the product's columns)
};
constexpr int tile_cols(int epi) { return epi == kGate ? 128 : 256; }

// Tile `t` of the launch: bands of 8 tiles of rows, column by column, so that the pairs that run at one
// time share rows and columns in the L2.
__device__ __forceinline__ GemmTile tile_of(const GemmArgs &g, int t, int cols) {
    if (g.back) t = g.tiles - 1 - t;
    GemmTile r;
    r.p = 0;
    while (r.p + 1 < g.problems && t >= g.count[r.p]) t -= g.count[r.p++];
    const int band = divide(t, g.band[r.p]), in = t - band * (int)g.band[r.p].d;
    int col, row;
    if (band < g.bands[r.p]) {
        col = in >> 3;
        row = in & 7;
    } else {
        col = divide(in, g.last[r.p]);
        row = in - col * (int)g.last[r.p].d;
    }
    r.row0 = (band * 8 + row) * 256;
    r.col0 = col * cols;
    return r;
}
// ... and the sizes that it goes by
inline long long place_tiles(GemmArgs &g, int cols) {
    long long n = 0;
    for (int p = 0; p < g.problems; ++p) {
        const int tm = (int)(((long long)g.M[p] + 255) / 256), tn = (g.N[p] + cols - 1) / cols;
        g.bands[p] = tm / 8;
        g.count[p] = tm * tn;
        g.band[p] = divisor((unsigned)(8 * tn));
        g.last[p] = divisor((unsigned)(tm % 8 ? tm % 8 : 1));
        n += (long long)tm * tn;
    }
    return n;
}

// ---- the epilogue's staging: a warp's box of 32 rows x 128 bytes ------------------------------

// 8 (bf16) or 4 (fp32) values to 16 bytes of a staged box
template <typename E>
__device__ __forceinline__ void stage(char *slab, int row, int piece, const float *x) {
    *reinterpret_cast<uint4 *>(slab + swz128(row, piece)) = Vec16<E>::pack(x);
}

// A warp's staged box to rows row .. and columns col .. of out [M, N], 128 bytes of four rows at a time; what lies
// outside is not written.  Plain stores of a box that is reused at once, instead of the TMA's out of four, leave room for
// a stage more of operands (16384 rows of 768 and 2048 channels: the gate 68 us, then 66; the products after it 39 and
// 37, the weights' gradients 84 and 82).
template <typename E>
__device__ __forceinline__ void store_box(const char *slab, void *out, int M, int N, int row, int col, int lane) {
    constexpr int PER = 16 / (int)sizeof(E);
    const int r = lane >> 3, p = lane & 7;
    E *to = static_cast<E *>(out) + (long long)(row + r) * N + col + p * PER;
    __syncwarp();
    if (col + p * PER < N) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row + r + 4 * i < M)
                __stcs(reinterpret_cast<uint4 *>(to + (long long)(4 * i) * N), *reinterpret_cast<const uint4 *>(slab + swz128(r + 4 * i, p)));
    }
    __syncwarp();  // the box may be filled again
}

// A warp's staged box by the TMA: fewer instructions, which counts in e4m3, where the MMAs wait for a tile's end (by
// plain stores the 8-bit product 66 us and the gated projection 300, by the TMA 61 and 278).
__device__ __forceinline__ void box_ready(int lane) {  // no box is being read
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
}
__device__ __forceinline__ void send_box(const char *slab, const void *map, bool inside, int row, int col, int lane) {
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
        store_3d(map, col, row, 0, slab);
        tc::bulk_commit();
    }
}

// ---- the kernel ------------------------------------------------------------------------------

struct GemmBars {
    uint64_t full[GST], empty[GST], acc_full[2], acc_empty[2], in[8][2];
    uint32_t tmem;
};

// What a warp of the epilogue knows of its place
struct EpiWarp {
    char *staging;
    uint64_t *in;   // its barriers for what the epilogue reads
    int lane, q, half, rank;  // 32 rows q, half of the columns, of two
    uint32_t tmem;            // of its lanes
};

// The accumulator has been read
__device__ __forceinline__ void release_acc(const EpiWarp &w, uint32_t release) {
    tc::tc_fence_before();
    __syncwarp();
    if (w.lane == 0) arrive_remote(release);
}

// Direct kind, kGate: columns c and 128 + c are the factors of the product's column c; 64 of them a warp.
__device__ __forceinline__ void epi_gate(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, uint32_t acc, uint32_t release) {
    using E = __nv_bfloat16;
    const int row = t.row0 + w.rank * 128 + w.q * 32, col = t.col0 + w.half * 64;
    uint32_t r[4][32];  // 64 of either factor
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32(acc + w.half * 64 + c / 2 * 128 + c % 2 * 32, r[c]);
    tc::tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_use(r[c]);
    release_acc(w, release);
    if (g.keep) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) stage<E>(w.staging, w.lane, k, reinterpret_cast<const float *>(r[2 * f + k / 4]) + k % 4 * 8);
            store_box<E>(w.staging, g.out[1 + f], g.M[0], g.N[0], row, col, w.lane);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float *xg = reinterpret_cast<const float *>(r[k / 4]) + k % 4 * 8, *xu = reinterpret_cast<const float *>(r[2 + k / 4]) + k % 4 * 8;
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = xg[e] * sigmoid<E>(xg[e]) * xu[e];
        stage<E>(w.staging, w.lane, k, h);
    }
    store_box<E>(w.staging, g.out[0], g.M[0], g.N[0], row, col, w.lane);
}

// d/dg and d/du of silu(g) u, given the product's gradient (u times the slope first, which is 1.1 at most: dh u may
// pass fp32 where the slope is 0)
template <typename E>
__device__ __forceinline__ void gate_grads(float dh, float &gate, float &up) {
    const float s = sigmoid<E>(gate), gs = gate * s;
    const float dg = dh * (up * (s + gs * (1.f - s)));
    up = dh * gs;
    gate = dg;
}

// Direct kind, kGateBwd: boxes of 32 columns (swizzled over 64 bytes) of both factors are read one box ahead
// (across tiles too), and the gradients written over them.
struct GateBwd {
    int n[2];  // uses of either pair of boxes
    __device__ __forceinline__ static bool inside(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, int j) {
        return t.row0 + w.rank * 128 + w.q * 32 < g.M[0] && t.col0 + w.half * 128 + j * 32 < g.N[0];
    }
    __device__ __forceinline__ static void ask(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, int j, int set) {
        if (w.lane != 0 || !inside(g, w, t, j)) return;
        char *s = w.staging + set * GSLAB;
        const int row = t.row0 + w.rank * 128 + w.q * 32, col = t.col0 + w.half * 128 + j * 32;
        bulk_wait_read<0>();  // the gradients that lay here have been stored
        tc::mbar_arrive_expect_tx(&w.in[set], GSLAB);
        load_3d(s, &g.e[0], col, row, 0, &w.in[set]);
        load_3d(s + GSLAB / 2, &g.e[1], col, row, 0, &w.in[set]);
    }
    // next: the tile behind this one (col0 < 0: none)
    __device__ __forceinline__ bool run(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, const GemmTile &next, uint32_t acc,
                                        uint32_t release) {
        using E = __nv_bfloat16;
        const int row = t.row0 + w.rank * 128 + w.q * 32;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const int set = j & 1;
            if (j < 3)
                ask(g, w, t, j + 1, set ^ 1);
            else if (next.col0 >= 0)
                ask(g, w, next, 0, set ^ 1);
            uint32_t r[32];
            tmem_ld32(acc + w.half * 128 + j * 32, r);
            tc::tmem_wait_ld();
            tmem_use(r);
            if (j == 3) release_acc(w, release);
            if (!inside(g, w, t, j)) continue;
            if (!pair_wait(&w.in[set], n[set]++ & 1, g.err)) return false;
            char *sg = w.staging + set * GSLAB, *su = sg + GSLAB / 2;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float xg[8], xu[8];
                const int at = w.lane * 64 + ((k ^ (w.lane >> 1 & 3)) << 4);
                Vec16<E>::unpack(*reinterpret_cast<const uint4 *>(sg + at), xg);
                Vec16<E>::unpack(*reinterpret_cast<const uint4 *>(su + at), xu);
#pragma unroll
                for (int e = 0; e < 8; ++e) gate_grads<E>(__uint_as_float(r[8 * k + e]), xg[e], xu[e]);
                *reinterpret_cast<uint4 *>(sg + at) = Vec16<E>::pack(xg);
                *reinterpret_cast<uint4 *>(su + at) = Vec16<E>::pack(xu);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (w.lane == 0) {
                store_3d(&g.o[0], t.col0 + w.half * 128 + j * 32, row, 0, sg);
                store_3d(&g.o[1], t.col0 + w.half * 128 + j * 32, row, 0, su);
                tc::bulk_commit();
            }
        }
        return true;
    }
};

// The other kinds: a thread's 128 sums of its row, in registers: half of the tile's columns, or (kGate) 64 of either
// factor.
template <int EPI>
__device__ __forceinline__ int sum_col(const EpiWarp &w, int c) {  // TMEM column of sums 16 c ..
    return EPI == kGate ? w.half * 64 + c / 4 * 128 + c % 4 * 16 : w.half * 128 + c * 16;
}

template <int KIND, int EPI, typename E>
__device__ __forceinline__ bool epi_sums(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, float (&x)[128], int &uses) {
    constexpr int BOX = 128 / (int)sizeof(E), PER = 16 / (int)sizeof(E);  // columns of a box, of a piece
    const int row = t.row0 + w.rank * 128 + w.q * 32;
    if constexpr (EPI == kPlain) {
        const int col = t.col0 + w.half * 128;
#pragma unroll
        for (int j = 0; j < 128 / BOX; ++j) {
            if (KIND == kE4M3) box_ready(w.lane);
#pragma unroll
            for (int k = 0; k < 8; ++k) stage<E>(w.staging, w.lane, k, x + j * BOX + k * PER);
            if (KIND == kE4M3)
                send_box(w.staging, &g.o[0], row < g.M[0] && col + j * BOX < g.N[0], row, col + j * BOX, w.lane);
            else
                store_box<E>(w.staging, g.out[t.p], g.M[t.p], g.N[t.p], row, col + j * BOX, w.lane);
        }
    } else if constexpr (EPI == kGate) {
        const int col = t.col0 + w.half * 64;
#pragma unroll
        for (int j = 0; j < 64 / BOX; ++j) {
            if (g.keep) {
#pragma unroll
                for (int f = 0; f < 2; ++f) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) stage<E>(w.staging, w.lane, k, x + f * 64 + j * BOX + k * PER);
                    store_box<E>(w.staging, g.out[1 + f], g.M[0], g.N[0], row, col + j * BOX, w.lane);
                }
            }
#pragma unroll
            for (int e = j * BOX; e < (j + 1) * BOX; ++e) x[e] = x[e] * sigmoid<E>(x[e]) * x[64 + e];
#pragma unroll
            for (int k = 0; k < 8; ++k) stage<E>(w.staging, w.lane, k, x + j * BOX + k * PER);
            store_box<E>(w.staging, g.out[0], g.M[0], g.N[0], row, col + j * BOX, w.lane);
        }
    } else {
        const int col = t.col0 + w.half * 128;
        char *sg = w.staging, *su = sg + GSLAB;
#pragma unroll
        for (int j = 0; j < 128 / BOX; ++j) {
            if (row >= g.M[0] || col + j * BOX >= g.N[0]) continue;
            if (w.lane == 0) {
                bulk_wait_read<0>();
                tc::mbar_arrive_expect_tx(w.in, 2 * GSLAB);
                load_3d(sg, &g.e[0], col + j * BOX, row, 0, w.in);
                load_3d(su, &g.e[1], col + j * BOX, row, 0, w.in);
            }
            if (!pair_wait(w.in, uses & 1, g.err)) return false;
            ++uses;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float xg[PER], xu[PER];
                const int at = swz128(w.lane, k);
                Vec16<E>::unpack(*reinterpret_cast<const uint4 *>(sg + at), xg);
                Vec16<E>::unpack(*reinterpret_cast<const uint4 *>(su + at), xu);
#pragma unroll
                for (int e = 0; e < PER; ++e) gate_grads<E>(x[j * BOX + k * PER + e], xg[e], xu[e]);
                *reinterpret_cast<uint4 *>(sg + at) = Vec16<E>::pack(xg);
                *reinterpret_cast<uint4 *>(su + at) = Vec16<E>::pack(xu);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (w.lane == 0) {
                store_3d(&g.o[0], col + j * BOX, row, 0, sg);
                store_3d(&g.o[1], col + j * BOX, row, 0, su);
                tc::bulk_commit();
            }
        }
    }
    return true;
}

// e4m3 values of quotients by a scale, rounded as a division rounds them, from its reciprocal: with r = 1 / d to the
// nearest and q within a unit of x / d, q + r (x - d q) in fused steps is x / d to the nearest (Markstein 1990), where
// no step underflows.  Quotients below 2^-10 are 0 in e4m3, so a scale of 2^-80 and more leaves the residual's
// bits above 2^-138; smaller ones are multiplied by 2^120 first, and the values with them, exactly.  All of it is negated
// until the values are in 8 bits: then a zero keeps its sign.  Two at a time.  (With divisions the quantiser of 4099
// rows of 5632 channels took 21 us, now 13.3, with four groups a thread instead of one.  By the reciprocal alone
// 14336 rows' gated projection would take 244 us, now 249, but of 768000 values made to lie at ties 8864 went the
// other way.)
struct Quotient {
    float up, d, nr;
    __device__ __forceinline__ explicit Quotient(float sc) {
        up = sc < 0x1p-80f ? 0x1p120f : 1.f;
        d = sc * up;
        nr = -1.f / d;
    }
    template <int N>
    __device__ __forceinline__ void scale_up(float (&x)[N], int n = N) const {  // before anything else
        if (up != 1.f) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e < n) x[e] *= up;
        }
    }
    __device__ __forceinline__ uint32_t two(float x0, float x1) const {  // still negated
        float n0, n1;
        asm("{\n\t.reg .b64 x, d, r, q, e;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 d, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
            "mul.rn.f32x2 q, x, r;\n\tfma.rn.f32x2 e, d, q, x;\n\tfma.rn.f32x2 e, r, e, q;\n\tmov.b64 {%0, %1}, e;\n\t}"
            : "=f"(n0), "=f"(n1)
            : "f"(x0), "f"(x1), "f"(d), "f"(nr));
        return __nv_cvt_float2_to_fp8x2(make_float2(n0, n1), __NV_SATFINITE, __NV_E4M3);
    }
    __device__ __forceinline__ uint32_t four(const float *x) const { return (two(x[0], x[1]) | two(x[2], x[3]) << 16) ^ 0x80808080u; }
    __device__ __forceinline__ uint8_t one(float x) const { return (uint8_t)(two(x * up, 0.f) ^ 0x80u); }
};
__device__ __forceinline__ float quant_scale(float top) {
    const float sc = top > 0.f ? top / 448.f : 1.f;
    return sc < 0x1p-126f ? __fdiv_ru(top, 448.f) : sc;
}

// kE4M3, kGate: the product's 64 columns of a thread, a scale for its row's 128 with the warp of the other half.
// Each warp's box is 32 rows of 64 bytes (swizzled over 64 bytes); behind it lie its rows' maxima for the other
// warp, which reads them once this one has arrived on its barrier (and before it arrives itself for the next
// tile, so that two sets are enough).  The barriers are two, taken in turn: a warp arrives before it waits, and
// with one the other might arrive again, for the next tile, before this one has seen that the phase it waits for is
// over; for tile n + 2 the other arrives behind its wait for n + 1, which ends when this one has waited for n.
// n: tiles before this one.
__device__ __forceinline__ bool epi_gate_e4m3(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, float (&x)[128], int n) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        gate_two(x[e], x[e + 1], x[64 + e], x[65 + e]);
        top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
    }
    char *slab = w.staging;
    box_ready(w.lane);
    const int at = GSLAB / 2 + (n & 1) * 128, other = w.half ? -4 : 4;  // warps to the other half's
    reinterpret_cast<float *>(slab + at)[w.lane] = top;
    __syncwarp();
    if (w.lane == 0) arrive_local(w.in + other * 2 + (n & 1));
    if (!pair_wait(w.in + (n & 1), n >> 1 & 1, g.err)) return false;
    top = fmaxf(top, reinterpret_cast<const float *>(slab + at + other * GSLAB)[w.lane]);
    const float sc = quant_scale(top);
    const Quotient by(sc);
    by.scale_up(x, 64);
    const int row = t.row0 + w.rank * 128 + w.q * 32, col = t.col0 + w.half * 64;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = by.four(x + 16 * k + 4 * e);
        *reinterpret_cast<uint4 *>(slab + w.lane * 64 + ((k ^ (w.lane >> 1 & 3)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    send_box(slab, &g.o[0], row < g.M[0] && col < g.N[0], row, col, w.lane);
    if (w.half == 0 && row + w.lane < g.M[0]) g.so[(size_t)(row + w.lane) * ((g.N[0] + 127) / 128) + t.col0 / 128] = sc;
    return true;
}

static_assert(sizeof(GemmBars) <= 512, "shared memory budget");

// Split products (kPlain of few tiles and a long contraction): a cluster of `split` pairs makes one tile, each pair a
// part of the contraction.  Each CTA lays its 128 x 256 fp32 sums where its operands were, [column / 4][row] so
// that a warp's 16-byte accesses lie side by side, and adds up its share of the columns over the pairs, in
// their order.  (256 rows of 5632 channels to 2048, eight tiles: 12 us in four parts, 28 in one.)
template <typename E>
__device__ __forceinline__ void add_parts(const GemmArgs &g, const EpiWarp &w, const GemmTile &t, const char *part, int group, int split) {
    const int r = w.q * 32 + w.lane, row = t.row0 + w.rank * 128 + r, own = (int)cluster_rank() >> 1;
    const int cols = 256 / split / (GEW / 4), c0 = own * (256 / split) + group * cols;
    if (row >= g.M[t.p]) return;
    E *out = static_cast<E *>(g.out[t.p]) + (long long)row * g.N[t.p] + t.col0;
    for (int c = c0; c < c0 + cols && t.col0 + c < g.N[t.p]; c += 8) {
        float x[8] = {};
        for (int p = 0; p < split; ++p) {
            const uint32_t from = cluster_addr(part + (c / 4 * 128 + r) * 16, 2 * p + w.rank);
            const float4 lo = cluster_float4(from), hi = cluster_float4(from + 128 * 16);
            x[0] += lo.x, x[1] += lo.y, x[2] += lo.z, x[3] += lo.w;
            x[4] += hi.x, x[5] += hi.y, x[6] += hi.z, x[7] += hi.w;
        }
#pragma unroll
        for (int k = 0; k < 8; k += Vec16<E>::n) *reinterpret_cast<uint4 *>(out + c + k) = Vec16<E>::pack(x + k);
    }
}

template <int AMN, int BMN, int KIND, int EPI, typename E, bool SPLIT>
__global__ void __launch_bounds__(gemm_threads(KIND), 1) gemm_kernel(const __grid_constant__ GemmArgs g) {
    constexpr bool E8 = KIND == kE4M3;
    constexpr int ST = gemm_stages(EPI), STAGING = gemm_staging(EPI);
    constexpr int EW = GEW, E0 = KIND == kDirect ? 2 : 4, COLS = tile_cols(EPI), KB = E8 ? 128 : 64;
    extern __shared__ char raw[];
    char *sm = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    char *ops = sm, *staging = sm + ST * 2 * GOP;
    GemmBars &bar = *reinterpret_cast<GemmBars *>(staging + STAGING);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, rank = (int)cluster_rank() & 1;
    const int tiles = g.tiles;
    // a split product's cluster makes one tile, any other pair every so many
    const int pair = SPLIT ? blockIdx.x / (2 * g.split) : blockIdx.x >> 1, pairs = SPLIT ? tiles : gridDim.x >> 1;
    const int all = g.segs * g.kblocks, part = SPLIT ? (int)cluster_rank() >> 1 : 0;
    const int kfirst = SPLIT ? all * part / g.split : 0, per_tile = (SPLIT ? all * (part + 1) / g.split : all) - kfirst;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&bar.full[s], 1);
            tc::mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&bar.acc_full[s], 1);
            tc::mbar_init(&bar.acc_empty[s], 2 * EW);
        }
        for (int s = 0; s < 2 * EW; ++s) tc::mbar_init(&bar.in[s >> 1][s & 1], 1);
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&bar.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    dependent_launch();
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc::tc_fence_after();
    const uint32_t tmem = bar.tmem;
    dependent_wait();

    // sums in registers: 168 of them a thread at launch (64512 in all), 40 for the first four warps leave
    // 232 for the other eight (64512)
    if (warp < E0) {
        if (KIND != kDirect) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        // These two roles' loops are run by whole warps and their waits end in a vote: the compiler then keeps
        // addresses and descriptors in uniform registers, where the one lane that issues wants them (moved there for
        // each instruction they held the MMAs up, 950 clocks a block of 512: 14336 rows' gated projection in 8 bits
        // 315 us, now 280; the block of 16384 rows in bf16 582, now 563).
        const bool one = tc::elect_one();
        if (warp == 0) {
            int st = 0, ph = 1, it = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                const GemmTile tile = tile_of(g, t, COLS);
                const int row = tile.row0 + rank * 128, col = EPI == kGate ? tile.col0 : tile.col0 + rank * 128;
                int s = SPLIT ? kfirst / g.kblocks : 0, kb = kfirst - s * g.kblocks;
                GemmSeg sg = g.seg[s];
                for (int k = 0; k < per_tile; ++k) {
                    const CUtensorMap *ma = &g.a[tile.p + sg.a], *mb = &g.b[EPI == kGate ? sg.b + rank : tile.p + sg.b];
                    if (!(ok = warp_wait(&bar.empty[st], ph, g.err))) break;
                    if (one) {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&bar.full[st], 4 * GOP);
                        char *A = ops + st * 2 * GOP, *B = A + GOP;
                        const uint32_t full = lead_addr(&bar.full[st]);
                        if (AMN) {
                            pair_load(A, ma, row, kb * 64, sg.ap, full);
                            pair_load(A + GOP / 2, ma, row + 64, kb * 64, sg.ap, full);
                        } else {
                            pair_load(A, ma, kb * KB, row, sg.ap, full);
                        }
                        if (BMN) {
                            pair_load(B, mb, col, kb * 64, sg.bp, full);
                            pair_load(B + GOP / 2, mb, col + 64, kb * 64, sg.bp, full);
                        } else {
                            pair_load(B, mb, kb * KB, col, sg.bp, full);
                        }
                    }
                    ++it;
                    if (++st == ST) st = 0, ph ^= 1;
                    if (++kb == g.kblocks && k + 1 < per_tile) {
                        kb = 0;
                        sg = g.seg[++s];
                    }
                }
            }
            // this CTA's shared memory and barriers are in use until its last stages have been read
            for (int k = it > ST ? it - ST : 0; k < it; ++k) {
                if (ok)
                    ok = warp_wait(&bar.empty[k % ST], k / ST & 1, g.err);
                else if (rank == 0)
                    warp_wait(&bar.full[k % ST], k / ST & 1, g.err);
            }
        }
        if (warp == 1 && rank == 0) {
            constexpr uint32_t id = tc::idesc(256, 256, E8 ? 0 : 1, E8 ? 0 : 1, AMN, BMN);
            int st = 0, ph = 0, ab = 0, aph = 1;
            bool ok = true;
            const uint32_t ops32 = tc::smem_u32(ops);
            for (int t = pair; ok && t < tiles; t += pairs) {
                for (int k0 = 0; ok && k0 < per_tile; k0 += g.chunk) {
                    const int n = per_tile - k0 < g.chunk ? per_tile - k0 : g.chunk;
                    for (int j = 0; ok && j < n; ++j) {
                        if (!(ok = warp_wait(&bar.full[st], ph, g.err))) break;
                        if (j == 0 && !(ok = warp_wait(&bar.acc_empty[ab], aph, g.err))) break;
                        tc::tc_fence_after();
                        const uint32_t A = ops32 + st * 2 * GOP, B = A + GOP;
                        const tc::SmemDesc da = pair_desc(A, AMN ? GOP / 2 : 16), db = pair_desc(B, BMN ? GOP / 2 : 16);
                        if (one) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                tc::SmemDesc a = da, b = db;
                                a.lo += k * (AMN ? 2048 : 32) >> 4;
                                b.lo += k * (BMN ? 2048 : 32) >> 4;
                                pair_mma<E8>(tmem + ab * 256, a, b, id, j > 0 || k > 0);
                            }
                            pair_commit(&bar.empty[st]);
                            if (j == n - 1) pair_commit(&bar.acc_full[ab]);
                        }
                        if (++st == ST) st = 0, ph ^= 1;
                    }
                    ab ^= 1;
                    aph ^= ab == 0;
                }
            }
        }
        __syncwarp();
    } else {
        if (KIND != kDirect) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        EpiWarp w;
        const int ew = warp - E0;
        w.lane = lane;
        w.q = warp & 3;
        w.half = ew >> 2;
        w.rank = rank;
        w.staging = staging + ew * (STAGING / EW);
        w.in = bar.in[ew];
        w.tmem = tmem + ((uint32_t)(w.q * 32) << 16);
        int ch = 0;
        bool ok = true;
        if constexpr (KIND == kDirect) {
            GateBwd back = {{0, 0}};
            if (EPI == kGateBwd && pair < tiles) GateBwd::ask(g, w, tile_of(g, pair, COLS), 0, 0);
            for (int t = pair; ok && t < tiles; t += pairs, ++ch) {
                const GemmTile tile = tile_of(g, t, COLS);
                const int ab = ch & 1;
                if (!(ok = pair_wait(&bar.acc_full[ab], ch >> 1 & 1, g.err))) break;
                tc::tc_fence_after();
                const uint32_t acc = w.tmem + ab * 256, release = lead_addr(&bar.acc_empty[ab]);
                if constexpr (EPI == kGate) epi_gate(g, w, tile, acc, release);
                if constexpr (EPI == kGateBwd) {
                    GemmTile next = {0, 0, -1};
                    if (t + pairs < tiles) next = tile_of(g, t + pairs, COLS);
                    ok = back.run(g, w, tile, next, acc, release);
                }
            }
        } else {
            int uses = 0;
            GemmTile tile;
            // the scales are read a block ahead, a tile's first ones before the epilogue of the one before it
            const float *sa = nullptr, *sb0 = nullptr, *sb1 = nullptr;
            float na = 0.f, n0 = 0.f, n1 = 0.f;
            auto scales = [&](int i) {
                na = sa ? sa[i] : 0.f;
                n0 = sb0 ? sb0[i] : 0.f;
                if (EPI == kGate) n1 = sb1 ? sb1[i] : 0.f;
            };
            auto open = [&](int t) {
                tile = tile_of(g, t, COLS);
                if constexpr (E8) {
                    const int row = tile.row0 + rank * 128 + w.q * 32 + lane;
                    const int blk = tile.col0 / 128 + (EPI == kGate ? 0 : w.half);
                    sa = row < g.M[tile.p] ? g.sa + (size_t)row * g.kblocks + kfirst : nullptr;
                    const bool in = blk * 128 < g.N[tile.p];
                    sb0 = in ? g.sb[0] + (size_t)blk * g.kblocks + kfirst : nullptr;
                    if (EPI == kGate) sb1 = in ? g.sb[1] + (size_t)blk * g.kblocks : nullptr;
                    scales(0);
                }
            };
            if (pair < tiles) open(pair);
            for (int t = pair; ok && t < tiles; t += pairs) {
                float x[128];
#pragma unroll
                for (int e = 0; e < 128; ++e) x[e] = 0.f;
                for (int k0 = 0, i = 0; k0 < per_tile; k0 += g.chunk, ++ch, ++i) {
                    const int ab = ch & 1;
                    const float m0 = E8 ? na * n0 : 1.f, m1 = E8 && EPI == kGate ? na * n1 : m0;
                    if (E8 && i + 1 < per_tile) scales(i + 1);
                    if (!(ok = pair_wait(&bar.acc_full[ab], ch >> 1 & 1, g.err))) break;
                    tc::tc_fence_after();
                    const uint32_t acc = w.tmem + ab * 256;
                    uint32_t r[8][16];
                    auto fetch = [&](int c) { tmem_ld16(acc + sum_col<EPI>(w, c), r[c]); };
                    auto add = [&](int c) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2)
                            add_scaled(x[c * 16 + e], x[c * 16 + e + 1], r[c][e], r[c][e + 1], EPI == kGate && c >= 4 ? m1 : m0);
                    };
                    // half of them; the others come while these are added, into the registers that they leave; and the
                    // accumulator is released before the last are added
#pragma unroll
                    for (int c = 0; c < 4; ++c) fetch(c);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_use(r[c]);
                    fetch(4);
                    add(0);
                    add(1);
                    fetch(5);
                    fetch(6);
                    add(2);
                    add(3);
                    fetch(7);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 4; c < 8; ++c) tmem_use(r[c]);
                    release_acc(w, lead_addr(&bar.acc_empty[ab]));
#pragma unroll
                    for (int c = 4; c < 8; ++c) add(c);
                }
                if (!ok) break;
                const GemmTile done = tile;
                if (t + pairs < tiles) open(t + pairs);
                if constexpr (SPLIT) {
#pragma unroll
                    for (int e = 0; e < 128; e += 4)
                        *reinterpret_cast<float4 *>(ops + ((w.half * 128 + e) / 4 * 128 + w.q * 32 + lane) * 16) =
                            make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                } else if constexpr (E8 && EPI == kGate)
                    ok = epi_gate_e4m3(g, w, done, x, uses++);
                else
                    ok = epi_sums<KIND, EPI, E>(g, w, done, x, uses);
            }
        }
        if ((EPI == kGateBwd || E8) && lane == 0) bulk_wait_read<0>();  // staging is read until then
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc::tc_fence_after();
    if constexpr (SPLIT) {
        if (warp >= E0) {
            EpiWarp w = {};
            w.lane = lane;
            w.q = warp & 3;
            w.rank = rank;
            add_parts<E>(g, w, tile_of(g, pair, COLS), ops, (warp - E0) >> 2, g.split);
        }
        __syncthreads();
        cluster_sync_all();  // the other pairs have read this one's sums
    }
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- host side ---------------------------------------------------------------------------------

ida_status device_error_word(unsigned **err, std::string &why);

enum { kMapBf16 = 0, kMapF32 = 1, kMapBytes = 2 };
// Rows of `inner` elements, ld bytes apart, in `parts` equal parts one behind the other; boxes of box0 x box1
// elements.  What lies outside is read as zero and not written.
ida_status gemm_map(CUtensorMap *m, const void *p, int type, long long inner, long long rows, int parts, long long ld, int box0,
                    int box1);

// Pairs to a tile: four or two where so many clusters fit the SMs at once (15 of eight CTAs, 36 of four on 152) and
// each part keeps eight blocks of the contraction.
inline int split_of(long long tiles, int blocks, int num_sms) {
    if (tiles * 10 <= num_sms && blocks >= 32) return 4;
    if (tiles * 9 <= 2 * num_sms && blocks >= 16) return 2;
    return 1;
}

template <int AMN, int BMN, int KIND, int EPI, typename E, bool SPLIT>
ida_status gemm_launch_as(GemmArgs &g, int num_sms, cudaStream_t st) {
    const auto kernel = gemm_kernel<AMN, BMN, KIND, EPI, E, SPLIT>;
    constexpr int smem = gemm_smem(EPI);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long pairs = SPLIT ? (long long)g.tiles * g.split : g.tiles < num_sms / 2 ? g.tiles : num_sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(gemm_threads(KIND));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = SPLIT ? 2 * g.split : 2;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, g);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("matrix product launch: ") + cudaGetErrorString(e));
    return launched("matrix product");
}

template <int AMN, int BMN, int KIND, int EPI, typename E>
ida_status gemm_launch(GemmArgs &g, int num_sms, cudaStream_t st) {
    const long long tiles = place_tiles(g, tile_cols(EPI));
    if (tiles > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many tiles");
    g.tiles = (int)tiles;
    if (KIND == kDirect) g.chunk = g.segs * g.kblocks;
    if constexpr (EPI == kPlain) {
        g.split = split_of(tiles, g.segs * g.kblocks, num_sms);
        if (g.split > 1) return gemm_launch_as<AMN, BMN, KIND, EPI, E, true>(g, num_sms, st);
    }
    return gemm_launch_as<AMN, BMN, KIND, EPI, E, false>(g, num_sms, st);
}

// The products by operand layout (a_mn, b_mn: the contraction is the outer dimension in memory) and epilogue.
ida_status gemm_bf16(int a_mn, int b_mn, int epi, GemmArgs &g, int num_sms, cudaStream_t st);
ida_status gemm_f32(int a_mn, int b_mn, int epi, GemmArgs &g, int num_sms, cudaStream_t st);

}  // namespace ida
