// ida_ssm_backward.cu -- the backward pass of the selective scan: its entry point, and its kernels on
// the CUDA cores (fp32 inputs, and the sizes ida_ssm_bwd_tc.cu does not take).
//
// With Z_t the adjoint of the state X_t (per row and head; see ida_ssm.cuh for the forward):
//   Z_t = c_t dy_t^T + a_{t+1} Z_{t+1},
//   dc_t = X_t dy_t,   db_t = D_t Z_t x_t,   dx_t = D_t Z_t^T b_t + D dy_t,
//   w_t  = <Z_t, a_t X_{t-1}>  (the gradient of log a_t),
//   dD_t = b_t^T Z_t x_t - e^{a_log} w_t,   ddt_t = dD_t / (1 + e^-z),  da_log = -e^{a_log} sum D_t w_t,
// db and dc summed over the heads of a group.  w needs no product of two states per position:
// <Z_t, X_t> is c_t^T X_t dy_t + w_{t+1} by Z's recurrence and w_t + D_t b_t^T Z_t x_t by X's, and
// without the term of position t itself that both hold,
//   w_t = w_{t+1} + c_t^T (a_t X_{t-1}) dy_t - D_t b_t^T (a_{t+1} Z_{t+1}) x_t,
// from the product of the two states at the end of t's group of 8 positions.  Groups are short so
// that this sum of differences loses little: its rounding is 2^-24 of the terms of one group.  (Over
// whole chunks it cost 4e-6 of a_log's gradient in heads that forget within a few positions.)
//
// Sequences are cut into chunks of 64 positions (32 where the rows would not fit shared memory).
// Launches: each chunk's last state from zero and, backwards, what it passes on of its own
// adjoint; the two running sums over the chunks; then every chunk by itself, a walk forwards
// from its first state for dc and one backwards from its last adjoint for dx and db, the state
// in registers as in the forward scan; the sums over the heads of a group and over chunks.
// All sums run in a fixed order.
#include "ida_ssm.cuh"

namespace ida {

ida_status check_scan(int B, int H, int N, int d, int G, int M, long long ldx, long long ldb, long long ldc,
                      long long lddt, int dtype);
ida_status device_error_word(unsigned **err, std::string &why);
int ssm_bwd_tc_chunk(int M);
int ssm_bwd_tc_splits(int B, int H, int N, int G, int M);
ida_status launch_bwd_tc_states(const ScanBwdArgs &a, cudaStream_t st);
ida_status launch_bwd_tc(const ScanBwdArgs &a, int splits, cudaStream_t st);

constexpr int BT = 8;  // positions between two sums across warps, and of a group (w above)

// floats of a quarter row of b or c and of a row (the four quarters on their own banks)
template <int MT>
struct BwdRow {
    static constexpr int QS = MT + 4, MS = 4 * QS;
};

// cols: columns of a CTA, a warp's 32 each, all of the head's.
template <int MT>
static size_t bwd_smem(int cols, int chunk) {
    return ((size_t)chunk * (2 * BwdRow<MT>::MS + 2 * cols) + 7 * (size_t)chunk + (size_t)(cols / 32) * BT * 4 * MT +
            64) * sizeof(float);
}

// The rows of one chunk in shared memory, as fp32.
template <typename E, int MT>
struct ChunkRows {
    float *b, *c, *x, *dy, *delta, *a, *z;  // z: dt + dt_bias
    __device__ __forceinline__ float *carve(float *p, int chunk, int cols) {
        b = p;
        c = b + chunk * BwdRow<MT>::MS;
        x = c + chunk * BwdRow<MT>::MS;
        dy = x + chunk * cols;
        delta = dy + chunk * cols;
        a = delta + chunk;
        z = a + chunk;
        return z + chunk;
    }
    // rows of positions t0 .. t0 + chunk, zero behind the end
    __device__ __forceinline__ void load(const ScanBwdArgs &s, int unit, int t0, int chunk, int cols, bool want_bx,
                                         bool want_cdy) {
        using V = Vec16<E>;
        const int M = s.M, d = s.d, H = s.H, N = s.N;
        const int bb = unit / H, h = unit % H, g = h / (H / s.G);
        const size_t row = (size_t)bb * N + t0;
        const int left = N - t0;
        const auto fill_bc = [&](const void *src, long long ld, float *dst) {
            const E *p = static_cast<const E *>(src) + row * ld + g * M;
            const int vpr = 4 * MT / V::n;
#pragma unroll 4
            for (int i = threadIdx.x; i < chunk * vpr; i += blockDim.x) {
                const int t = i / vpr, m = i % vpr * V::n;
                float v[V::n];
                uint4 u = make_uint4(0, 0, 0, 0);
                if (t < left && m < M) u = __ldg(reinterpret_cast<const uint4 *>(p + (size_t)t * ld + m));
                V::unpack(u, v);
#pragma unroll
                for (int k = 0; k < V::n; ++k)
                    dst[t * BwdRow<MT>::MS + (m + k) / MT * BwdRow<MT>::QS + (m + k) % MT] = v[k];
            }
        };
        const auto fill_x = [&](const void *src, size_t at, long long ld, float *dst) {
            const E *p = static_cast<const E *>(src) + at;
            const int vpr = cols / V::n;
#pragma unroll 4
            for (int i = threadIdx.x; i < chunk * vpr; i += blockDim.x) {
                const int t = i / vpr, j = i % vpr * V::n;
                float v[V::n];
                uint4 u = make_uint4(0, 0, 0, 0);
                if (t < left && j < d) u = __ldg(reinterpret_cast<const uint4 *>(p + (size_t)t * ld + j));
                V::unpack(u, v);
#pragma unroll
                for (int k = 0; k < V::n; ++k) dst[t * cols + j + k] = v[k];
            }
        };
        if (want_bx) {
            fill_bc(s.b, s.ldb, b);
            fill_x(s.x, row * s.ldx + (size_t)h * d, s.ldx, x);
        }
        if (want_cdy) {
            fill_bc(s.c, s.ldc, c);
            fill_x(s.dy, (row * H + h) * d, (long long)H * d, dy);
        }
        const float rate = scan_rate(s.a_log[h]), bias = s.dt_bias[h];
        for (int t = threadIdx.x; t < chunk; t += blockDim.x) {
            float dl = 0.f, zz = 0.f;
            if (t < left) {
                zz = to_float(static_cast<const E *>(s.dt)[(row + t) * s.lddt + h]) + bias;
                dl = softplus(zz);
            }
            delta[t] = dl;
            z[t] = zz;
            a[t] = expf(-rate * dl);
        }
    }
};

// The state tile's step X <- a X + u x over a lane's rows and four columns, in its two parts.
template <int MT>
__device__ __forceinline__ void tile_scale(ssm_f2 (&X)[MT / 2][4], float a) {
    const ssm_f2 aa = ssm_pack(a, a);
#pragma unroll
    for (int i = 0; i < MT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) X[i][j] = ssm_mul(aa, X[i][j]);
}
template <int MT>
__device__ __forceinline__ void tile_add(ssm_f2 (&X)[MT / 2][4], const float *u, float f, float4 x) {
    const ssm_f2 xx[4] = {ssm_pack(f * x.x, f * x.x), ssm_pack(f * x.y, f * x.y), ssm_pack(f * x.z, f * x.z),
                          ssm_pack(f * x.w, f * x.w)};
#pragma unroll
    for (int i = 0; i < MT / 2; i += 2) {
        const ulonglong2 u2 = *reinterpret_cast<const ulonglong2 *>(u + 2 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            X[i][j] = ssm_fma(u2.x, xx[j], X[i][j]);
            X[i + 1][j] = ssm_fma(u2.y, xx[j], X[i + 1][j]);
        }
    }
}

// Rows of the state tile times four columns' values, summed over the warp's columns (the lanes of
// equal l % 4): *out [4 MT] receives the sums, quarter by quarter.
template <int MT>
__device__ __forceinline__ void tile_rows(const ssm_f2 (&X)[MT / 2][4], float4 v, int lane, float *out) {
    const ssm_f2 vv[4] = {ssm_pack(v.x, v.x), ssm_pack(v.y, v.y), ssm_pack(v.z, v.z), ssm_pack(v.w, v.w)};
    float s[MT];
#pragma unroll
    for (int i = 0; i < MT / 2; ++i) {
        ssm_f2 t = ssm_mul(X[i][0], vv[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) t = ssm_fma(X[i][j], vv[j], t);
        ssm_unpack(t, s[2 * i], s[2 * i + 1]);
    }
    // recursive halving over lane bits 4, 3, 2; with MT = 4 the last step adds both halves
    int n = MT, base = 0;
#pragma unroll
    for (int off = 16; off >= 4; off >>= 1) {
        const bool up = (lane & off) != 0;
        if (n > 1) {
            const int hn = n >> 1;
#pragma unroll
            for (int k = 0; k < MT / 2; ++k)
                if (k < hn) {
                    const float send = up ? s[k] : s[k + hn], keep = up ? s[k + hn] : s[k];
                    s[k] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                }
            if (up) base += hn;
            n = hn;
        } else {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
        }
    }
#pragma unroll
    for (int k = 0; k < (MT / 8 > 0 ? MT / 8 : 1); ++k) out[(lane & 3) * MT + base + k] = s[k];
}

// Columns of the state tile times the rows' values: lane l receives column l of the warp.
template <int MT>
__device__ __forceinline__ float tile_cols(const ssm_f2 (&X)[MT / 2][4], const float *u, int lane) {
    ssm_f2 acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int i = 0; i < MT / 2; i += 2) {
        const ulonglong2 u2 = *reinterpret_cast<const ulonglong2 *>(u + 2 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = ssm_fma(u2.x, X[i][j], acc[j]);
            acc[j] = ssm_fma(u2.y, X[i + 1][j], acc[j]);
        }
    }
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float lo, hi;
        ssm_unpack(acc[j], lo, hi);
        y[j] = lo + hi;
    }
    const bool up = (lane & 2) != 0, odd = (lane & 1) != 0;
    const float k0 = (up ? y[2] : y[0]) + __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 2);
    const float k1 = (up ? y[3] : y[1]) + __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 2);
    return (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
}

// Chunk c of a unit, by itself: blockIdx.y 0 leaves its last state from zero in state0[c], 1 what
// it passes on of its own adjoint, sum_t a_first .. a_t c_t dy_t^T, in adj[c].
template <typename E, int MT>
__global__ void __launch_bounds__(256) bwd_chunk_kernel(ScanBwdArgs s) {
    dependent_launch();
    extern __shared__ __align__(16) float sm[];
    const int M = s.M, d = s.d, Q = s.chunk, cols = (d + 31) / 32 * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / s.chunks, ch = blockIdx.x % s.chunks;
    const bool rev = blockIdx.y != 0;
    ChunkRows<E, MT> r;
    r.carve(sm, Q, cols);
    r.load(s, unit, ch * Q, Q, cols, !rev, rev);
    __syncthreads();
    const int km = lane & 3, jl = warp * 32 + (lane >> 2) * 4, ms = BwdRow<MT>::MS, qs = BwdRow<MT>::QS;
    const int len = min(Q, s.N - ch * Q);
    if (warp < cols / 32) {  // the others have helped to load
    ssm_f2 X[MT / 2][4];
#pragma unroll
    for (int i = 0; i < MT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) X[i][j] = 0ull;
    if (!rev) {
        for (int t = 0; t < len; ++t) {
            tile_scale<MT>(X, r.a[t]);
            tile_add<MT>(X, r.b + t * ms + km * qs, r.delta[t], *reinterpret_cast<const float4 *>(r.x + t * cols + jl));
        }
    } else {
        for (int t = len - 1; t >= 0; --t) {
            tile_add<MT>(X, r.c + t * ms + km * qs, 1.f, *reinterpret_cast<const float4 *>(r.dy + t * cols + jl));
            tile_scale<MT>(X, r.a[t]);
        }
    }
    float *out = (rev ? s.adj : s.state0) + ((size_t)unit * s.chunks + ch) * M * d;
    if (jl < d)
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
            const int m = km * MT + 2 * i;
            if (m < M) {
                float u[4], v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ssm_unpack(X[i][j], u[j], v[j]);
                *reinterpret_cast<float4 *>(out + (size_t)m * d + jl) = make_float4(u[0], u[1], u[2], u[3]);
                *reinterpret_cast<float4 *>(out + (size_t)(m + 1) * d + jl) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    }
    if (!rev && warp == (int)blockDim.x / 32 - 1) {
        float la = 0.f;
        const float rate = scan_rate(s.a_log[unit % s.H]) * 1.4426950408889634f;
        for (int t = lane; t < Q; t += 32) la -= rate * r.delta[t];
        la = warp_sum(la);
        if (lane == 0) s.chunk_log[(size_t)unit * s.chunks + ch] = la;
    }
}

// The running sums over the chunks, in place: state0[c] becomes the state before chunk c, adj[c]
// what reaches chunk c from behind.  One thread per four state elements.
__global__ void __launch_bounds__(256) bwd_carry_kernel(ScanBwdArgs s) {
    dependent_launch();
    dependent_wait();
    const int unit = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x, n = s.M * s.d / 4;
    if (i >= n) return;
    const bool rev = blockIdx.z != 0;
    float4 *p = reinterpret_cast<float4 *>((rev ? s.adj : s.state0) + (size_t)unit * s.chunks * s.M * s.d) + i;
    const float *lg = s.chunk_log + (size_t)unit * s.chunks;
    float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int K = 8;
    for (int k0 = 0; k0 < s.chunks; k0 += K) {
        float4 v[K];
        float f[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k0 + k < s.chunks) {
                const int c = rev ? s.chunks - 1 - (k0 + k) : k0 + k;
                v[k] = p[(size_t)c * n];
                f[k] = lg[c];
            }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k0 + k < s.chunks) {
                const int c = rev ? s.chunks - 1 - (k0 + k) : k0 + k;
                p[(size_t)c * n] = X;
                const float e = exp2f(f[k]);
                X = make_float4(fmaf(e, X.x, v[k].x), fmaf(e, X.y, v[k].y), fmaf(e, X.z, v[k].z), fmaf(e, X.w, v[k].w));
            }
    }
}

template <typename E, int MT>
__global__ void __launch_bounds__(256) bwd_main_kernel(ScanBwdArgs s) {
    dependent_launch();
    dependent_wait();
    extern __shared__ __align__(16) float sm[];
    const int M = s.M, d = s.d, Q = s.chunk, H = s.H, N = s.N, cols = (d + 31) / 32 * 32;
    // the first `warps` warps walk the positions, all load and sum
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = cols / 32, all_warps = blockDim.x / 32;
    const bool walks = warp < warps;
    const int unit = blockIdx.x / s.chunks, ch = blockIdx.x % s.chunks, b = unit / H, h = unit % H;
    const int t0 = ch * Q, len = min(Q, N - t0);
    constexpr int MS = BwdRow<MT>::MS, QS = BwdRow<MT>::QS, MP = 4 * MT;
    ChunkRows<E, MT> r;
    float *p = r.carve(sm, Q, cols);
    float *pw = p;          // [Q]: c_t^T (a_t X_{t-1}) dy_t
    float *rw = pw + Q;     // [Q]: b_t^T (a_{t+1} Z_{t+1}) x_t
    float *xdy = rw + Q;    // [Q]: x_t . dy_t
    float *bc = xdy + Q;    // [Q]: b_t . c_t
    float *rows = bc + Q;                    // [warps][BT][4 MT]
    float *misc = rows + warps * BT * MP;    // [64]
    r.load(s, unit, t0, Q, cols, true, true);
    const int km = lane & 3, jl = warp * 32 + (lane >> 2) * 4, col = warp * 32 + lane;
    const size_t so = ((size_t)unit * s.chunks + ch) * M * d;
    ssm_f2 X[MT / 2][4];
    const auto load_tile = [&](const float *src, bool product) {  // product: with the tile that was there
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
            const int m = km * MT + 2 * i;
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
            if (m < M && jl < d) {
                u = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)m * d + jl));
                v = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)(m + 1) * d + jl));
            }
            if (product) {
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ssm_unpack(X[i][j], x[j], y[j]);
                dot += x[0] * u.x + x[1] * u.y + x[2] * u.z + x[3] * u.w + y[0] * v.x + y[1] * v.y + y[2] * v.z + y[3] * v.w;
            }
            X[i][0] = ssm_pack(u.x, v.x);
            X[i][1] = ssm_pack(u.y, v.y);
            X[i][2] = ssm_pack(u.z, v.z);
            X[i][3] = ssm_pack(u.w, v.w);
        }
        return dot;
    };
    // the state behind a group of BT, kept for the walk backwards
    float *kept = s.kept + ((size_t)unit * s.chunks + ch) * (Q / BT) * M * d;
    const auto keep_tile = [&](float *dst) {
        if (jl < d)
#pragma unroll
            for (int i = 0; i < MT / 2; ++i) {
                const int m = km * MT + 2 * i;
                if (m < M) {
                    float u[4], v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) ssm_unpack(X[i][j], u[j], v[j]);
                    *reinterpret_cast<float4 *>(dst + (size_t)m * d + jl) = make_float4(u[0], u[1], u[2], u[3]);
                    *reinterpret_cast<float4 *>(dst + (size_t)(m + 1) * d + jl) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
    };
    const auto kept_product = [&](const float *src) {  // of this thread's own part
        float dot = 0.f;
        if (jl < d)
#pragma unroll
            for (int i = 0; i < MT / 2; ++i) {
                const int m = km * MT + 2 * i;
                if (m < M) {
                    const float4 u = *reinterpret_cast<const float4 *>(src + (size_t)m * d + jl);
                    const float4 v = *reinterpret_cast<const float4 *>(src + (size_t)(m + 1) * d + jl);
                    float x[4], y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) ssm_unpack(X[i][j], x[j], y[j]);
                    dot += x[0] * u.x + x[1] * u.y + x[2] * u.z + x[3] * u.w + y[0] * v.x + y[1] * v.y + y[2] * v.z + y[3] * v.w;
                }
            }
        return dot;
    };
    if (walks) load_tile(s.state0 + so, false);
    __syncthreads();
    for (int t = warp; t < len; t += all_warps) {  // the products of a position with itself
        float v = 0.f, u = 0.f;
        for (int j = lane; j < cols; j += 32) v = fmaf(r.x[t * cols + j], r.dy[t * cols + j], v);
        for (int m = lane; m < M; m += 32) {
            const int at = t * MS + m / MT * QS + m % MT;
            u = fmaf(r.b[at], r.c[at], u);
        }
        v = warp_sum(v);
        u = warp_sum(u);
        if (lane == 0) {
            xdy[t] = v;
            bc[t] = u;
        }
    }

    // One head's rows of dc (is_c) or db: the sum over its warps plus the position's own term.
    // `dots` receives the sum's product with the position's c or b.
    const auto flush_rows = [&](int tb, int nb, bool is_c, float *dots) {
        __syncthreads();
        float *head = is_c ? s.dc_head : s.db_head;
        for (int tt = warp; tt < nb; tt += all_warps) {
            const int t = tb + tt;
            const float delta = r.delta[t], self = xdy[t] * delta, f = is_c ? 1.f : delta;
            float dot = 0.f;
            for (int m = lane; m < M; m += 32) {
                float o = 0.f;
                for (int w = 0; w < warps; ++w) o += rows[(w * BT + tt) * MP + m];
                const int i = t * MS + m / MT * QS + m % MT;
                const float bm = r.b[i], cm = r.c[i];
                dot = fmaf(o, is_c ? cm : bm, dot);
                o = fmaf(o, f, self * (is_c ? bm : cm));
                const size_t at = ((size_t)b * N + t0 + t);
                if (head)
                    head[(at * H + h) * M + m] = o;
                else
                    from_float(static_cast<E *>(is_c ? s.dc : s.db) + at * (is_c ? s.lddc : s.lddb) + (size_t)h * M + m, o);
            }
            dot = warp_sum(dot);
            if (lane == 0) dots[t] = dot;
        }
        __syncthreads();
    };

    // forwards: a_t X_{t-1} for dc_t, then X_t
    for (int tb = 0; tb < len; tb += BT) {
        const int nb = min(BT, len - tb);
        for (int tt = 0; walks && tt < nb; ++tt) {
            const int t = tb + tt;
            tile_scale<MT>(X, r.a[t]);
            tile_rows<MT>(X, *reinterpret_cast<const float4 *>(r.dy + t * cols + jl), lane, rows + (warp * BT + tt) * MP);
            tile_add<MT>(X, r.b + t * MS + km * QS, r.delta[t], *reinterpret_cast<const float4 *>(r.x + t * cols + jl));
        }
        flush_rows(tb, nb, true, pw);
        if (walks && tb + BT < len) keep_tile(kept + (size_t)(tb / BT) * M * d);
    }
    // w behind a group: <a Z of the next position, X of the last>; here the chunk's last group
    const float end = walks ? warp_sum(load_tile(s.adj + so, true)) : 0.f;
    if (walks && lane == 0) misc[(len - 1) / BT * 8 + warp] = end;

    // backwards: a_{t+1} Z_{t+1} for db_t and dx_t, then Z_t
    const float skip = s.D[h];
    for (int tb = (len - 1) / BT * BT; tb >= 0; tb -= BT) {
        const int nb = min(BT, len - tb);
        if (walks && tb + BT < len) {
            const float v = warp_sum(kept_product(kept + (size_t)(tb / BT) * M * d));
            if (lane == 0) misc[tb / BT * 8 + warp] = v;
        }
        for (int tt = nb - 1; walks && tt >= 0; --tt) {
            const int t = tb + tt;
            tile_rows<MT>(X, *reinterpret_cast<const float4 *>(r.x + t * cols + jl), lane, rows + (warp * BT + tt) * MP);
            const float o = tile_cols<MT>(X, r.b + t * MS + km * QS, lane), gv = r.dy[t * cols + col];
            tile_add<MT>(X, r.c + t * MS + km * QS, 1.f, *reinterpret_cast<const float4 *>(r.dy + t * cols + jl));
            tile_scale<MT>(X, r.a[t]);
            if (col < d)
                from_float(static_cast<E *>(s.dx) + ((size_t)b * N + t0 + t) * s.lddx + (size_t)h * d + col,
                           fmaf(r.delta[t], fmaf(bc[t], gv, o), skip * gv));
        }
        flush_rows(tb, nb, false, rw);
    }
    // w, and the gradients of dt and of the head's parameters: one warp, two positions a lane
    if (warp == 0) {
        const float rate = scan_rate(s.a_log[h]);
        float ga = 0.f, gb = 0.f, gd = 0.f;
        for (int base = 0; base < len; base += 32) {
            const int t = base + lane;
            const bool ok = t < len;
            float w = ok ? pw[t] - r.delta[t] * rw[t] : 0.f;
#pragma unroll
            for (int o = 1; o < BT; o <<= 1) {  // sum of the group's positions from mine on
                const float u = __shfl_down_sync(0xffffffffu, w, o);
                if ((lane & (BT - 1)) + o < BT) w += u;
            }
            if (ok)
                for (int i = 0; i < warps; ++i) w += misc[t / BT * 8 + i];
            if (ok) {
                const float sig = 1.f / (1.f + expf(-r.z[t]));
                const float ddt = (fmaf(bc[t], xdy[t], rw[t]) - rate * w) * sig;
                from_float(static_cast<E *>(s.ddt) + ((size_t)b * N + t0 + t) * s.ldddt + h, ddt);
                ga -= rate * (r.delta[t] * w);  // 0 where w is, whatever the rate
                gb += ddt;
                gd += xdy[t];
            }
        }
        ga = warp_sum(ga);
        gb = warp_sum(gb);
        gd = warp_sum(gd);
        if (lane == 0) *reinterpret_cast<float4 *>(s.part + ((size_t)unit * s.chunks + ch) * 4) = make_float4(ga, gb, gd, 0.f);
    }
}

// db and dc of a group: the sum over the `n` parts its heads were taken in, in their order.  One
// thread per four channels.
template <typename E>
__global__ void __launch_bounds__(256) bwd_group_kernel(ScanBwdArgs s, int n) {
    dependent_launch();
    dependent_wait();
    const int vpr = s.G * s.M / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)s.B * s.N * vpr) return;
    const long long row = i / vpr;
    const int v = (int)(i % vpr), g = v / (s.M / 4), m = v % (s.M / 4) * 4;
    const float *src = (blockIdx.y ? s.dc_head : s.db_head) + ((size_t)row * s.G + g) * n * s.M + m;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(src + (size_t)r * s.M));
        o.x += u.x;
        o.y += u.y;
        o.z += u.z;
        o.w += u.w;
    }
    E *dst = static_cast<E *>(blockIdx.y ? s.dc : s.db) + (size_t)row * (blockIdx.y ? s.lddc : s.lddb) + (size_t)g * s.M + m;
    from_float(dst, o.x);
    from_float(dst + 1, o.y);
    from_float(dst + 2, o.z);
    from_float(dst + 3, o.w);
}

// The head's parameter gradients: its chunks' parts over all rows, 128 interleaved sums.
__global__ void __launch_bounds__(128) bwd_params_kernel(ScanBwdArgs s, int per) {  // per: parts of a chunk
    __shared__ float red[4][3];
    dependent_wait();
    const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v[3] = {0.f, 0.f, 0.f};
    const long long n = (long long)s.B * s.chunks * per;
    for (long long i = threadIdx.x; i < n; i += 128) {
        const long long b = i / (s.chunks * per), c = i % (s.chunks * per);
        const float4 u = *reinterpret_cast<const float4 *>(s.part + ((size_t)(b * s.H + h) * s.chunks * per + c) * 4);
        v[0] += u.x;
        v[1] += u.y;
        v[2] += u.z;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = warp_sum(v[k]);
        if (lane == 0) red[warp][k] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        const float o = red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x];
        (threadIdx.x == 0 ? s.da_log : threadIdx.x == 1 ? s.ddt_bias : s.dD)[h] = o;
    }
}

static int bwd_cols(int d) { return (d + 31) / 32 * 32; }
static int bwd_mt(int M) { return M <= 16 ? 4 : M <= 32 ? 8 : M <= 64 ? 16 : 32; }

// Positions per chunk: 64, or 32 where 64 rows of b, c, x and dy do not fit shared memory.
static int bwd_chunk_len(int d, int M) {
    const size_t floats = 64 * (size_t)(2 * (4 * bwd_mt(M) + 16) + 2 * bwd_cols(d) + 7) +
                          (size_t)bwd_cols(d) / 32 * BT * 4 * bwd_mt(M) + 64;
    return floats * 4 <= 220 * 1024 ? 64 : 32;
}

struct BwdPlan {
    bool tc;
    int chunk, chunks, parts;                      // parts: those a group's db and dc are summed from
    size_t state0, adj, kept, log, db, dc, part, total;  // float offsets
};
static BwdPlan bwd_plan(int B, int H, int N, int d, int G, int M, int dtype) {
    BwdPlan p;
    p.tc = dtype == IDA_BF16 && d <= 128;
    p.chunk = p.tc ? ssm_bwd_tc_chunk(M) : bwd_chunk_len(d, M);
    p.chunks = (N + p.chunk - 1) / p.chunk;
    p.parts = p.tc ? ssm_bwd_tc_splits(B, H, N, G, M) : H / G;
    const size_t units = (size_t)B * H, states = units * p.chunks * M * d;
    const size_t heads = p.parts == 1 ? 0 : (size_t)B * N * G * p.parts * M;
    p.state0 = 0;
    p.adj = p.state0 + states;
    p.kept = p.adj + states;
    p.db = p.kept + (p.tc ? 0 : states * (p.chunk / BT));
    p.dc = p.db + heads;
    p.part = p.dc + heads;
    p.log = p.part + units * p.chunks * (p.tc ? 16 : 4);
    p.total = p.log + (units * p.chunks + 3) / 4 * 4;
    return p;
}

// The running sums over the chunks: a launch per 65535 units.
static ida_status launch_bwd_carry(const ScanBwdArgs &s, cudaStream_t st) {
    for (int u0 = 0; u0 < s.B * s.H; u0 += 65535) {
        ScanBwdArgs t = s;
        t.state0 += (size_t)u0 * s.chunks * s.M * s.d;
        t.adj += (size_t)u0 * s.chunks * s.M * s.d;
        t.chunk_log += (size_t)u0 * s.chunks;
        const int units = s.B * s.H - u0 < 65535 ? s.B * s.H - u0 : 65535;
        const cudaError_t e = launch_dependent(bwd_carry_kernel, dim3((s.M * s.d / 4 + 255) / 256, units, 2), dim3(256), 0, st, t);
        if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm chunk sums launch: ") + cudaGetErrorString(e));
    }
    return IDA_OK;
}

// The sums over a group's parts and over the chunks.
template <typename E>
static ida_status launch_bwd_sums(const ScanBwdArgs &s, int parts, int per, cudaStream_t st) {
    if (s.db_head) {
        const long long n = ((long long)s.B * s.N * s.G * s.M / 4 + 255) / 256;
        const cudaError_t e = launch_dependent(bwd_group_kernel<E>, dim3((unsigned)n, 2), dim3(256), 0, st, s, parts);
        if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm group sums launch: ") + cudaGetErrorString(e));
    }
    const cudaError_t e = launch_dependent(bwd_params_kernel, dim3(s.H), dim3(128), 0, st, s, per);
    return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, std::string("ssm parameter gradients launch: ") + cudaGetErrorString(e));
}

template <typename E, int MT>
static ida_status launch_bwd(const ScanBwdArgs &s, cudaStream_t st) {
    // narrow heads get warps that help to load and to sum (32 channels: 121 us with one warp, 64 chunks)
    const int cols = bwd_cols(s.d), threads = cols + 128 < 256 ? cols + 128 : 256;
    const size_t smem = bwd_smem<MT>(cols, s.chunk);
    cudaError_t e = allow_smem(bwd_chunk_kernel<E, MT>, smem);
    if (e == cudaSuccess) e = allow_smem(bwd_main_kernel<E, MT>, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    const long long blocks = (long long)s.B * s.H * s.chunks;
    bwd_chunk_kernel<E, MT><<<dim3((unsigned)blocks, 2), threads, smem, st>>>(s);
    ida_status r = launched("ssm chunk states");
    if (r == IDA_OK) r = launch_bwd_carry(s, st);
    if (r != IDA_OK) return r;
    e = launch_dependent(bwd_main_kernel<E, MT>, dim3((unsigned)blocks), dim3(threads), smem, st, s);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, std::string("ssm scan backward launch: ") + cudaGetErrorString(e));
    return launch_bwd_sums<E>(s, s.H / s.G, 1, st);
}

template <typename E>
static ida_status launch_bwd_m(const ScanBwdArgs &s, cudaStream_t st) {
    switch (bwd_mt(s.M)) {
        case 4: return launch_bwd<E, 4>(s, st);
        case 8: return launch_bwd<E, 8>(s, st);
        case 16: return launch_bwd<E, 16>(s, st);
        default: return launch_bwd<E, 32>(s, st);
    }
}

}  // namespace ida

extern "C" {

size_t ida_ssm_scan_backward_workspace_bytes(int B, int H, int N, int d, int G, int M, int dtype) {
    using namespace ida;
    if (check_scan(B, H, N, d, G, M, (long long)H * d, (long long)G * M, (long long)G * M, H, dtype) != IDA_OK) return 0;
    if ((long long)B * H * N == 0) return 0;
    return bwd_plan(B, H, N, d, G, M, dtype).total * sizeof(float);
}

ida_status ida_ssm_scan_backward(const void *x, const void *b, const void *c, const void *dt, const float *a_log,
                                 const float *dt_bias, const float *D, const void *dy, void *dx, void *db, void *dc,
                                 void *ddt, float *da_log, float *ddt_bias, float *dD, int B, int H, int N, int d,
                                 int G, int M, long long ldx, long long ldb, long long ldc, long long lddt,
                                 long long lddx, long long lddb, long long lddc, long long ldddt, int dtype,
                                 void *workspace,
                                 size_t workspace_bytes, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_scan(B, H, N, d, G, M, ldx, ldb, ldc, lddt, dtype);
    if (s == IDA_OK) s = check_scan(B, H, N, d, G, M, lddx, lddb, lddc, ldddt, dtype);
    if (s != IDA_OK) return s;
    if (H == 0) return IDA_OK;
    if (!da_log || !ddt_bias || !dD) return fail_with(IDA_ERR_ARG, "null gradient pointer");
    if (misaligned4(da_log) || misaligned4(ddt_bias) || misaligned4(dD))
        return fail_with(IDA_ERR_ARG, "da_log, ddt_bias and dD must be 4-byte aligned");
    const bool work = B > 0 && N > 0;
    if (work) {
        const void *ptrs[] = {x, b, c, a_log, dt_bias, D, dy, dx, db, dc, workspace};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input, output or workspace pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        const void *narrow[] = {dt, ddt};
        for (const void *p : narrow)
            if (!p || (reinterpret_cast<uintptr_t>(p) % (dtype == IDA_F32 ? 4 : 2)))
                return fail_with(IDA_ERR_ARG, "dt and ddt must be aligned pointers");
        if (workspace_bytes < ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, dtype))
            return fail_with(IDA_ERR_ARG, "workspace is smaller than ida_ssm_scan_backward_workspace_bytes");
    }
    const long long n = (long long)B * N, w = (long long)H * d, bc = (long long)G * M;
    const size_t par = (size_t)H * 4;
    const Rows outs[] = {rows_of("dx", dx, lddx, w, n, dtype), rows_of("db", db, lddb, bc, n, dtype), rows_of("dc", dc, lddc, bc, n, dtype),
                         rows_of("ddt", ddt, ldddt, H, n, dtype), dense("da_log", da_log, par), dense("ddt_bias", ddt_bias, par),
                         dense("dD", dD, par),
                         dense("workspace", workspace, ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, dtype))};
    const Rows ins[] = {rows_of("x", x, ldx, w, n, dtype), rows_of("b", b, ldb, bc, n, dtype), rows_of("c", c, ldc, bc, n, dtype),
                        rows_of("dt", dt, lddt, H, n, dtype), rows_of("dy", dy, w, w, n, dtype), dense("a_log", work ? a_log : nullptr, par),
                        dense("dt_bias", work ? dt_bias : nullptr, par), dense("D", work ? D : nullptr, par)};
    s = check_overlaps(outs, ins);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!work) {
        cudaError_t e = cudaMemsetAsync(da_log, 0, H * sizeof(float), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(ddt_bias, 0, H * sizeof(float), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dD, 0, H * sizeof(float), st);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    }
    const BwdPlan p = bwd_plan(B, H, N, d, G, M, dtype);
    if ((long long)B * H * p.chunks > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many positions and heads");
    float *ws = static_cast<float *>(workspace);
    ScanBwdArgs a = {x, b, c, dt, dy, a_log, dt_bias, D, dx, db, dc, ddt, da_log, ddt_bias, dD, B, H, N, d, G, M,
                     ldx, ldb, ldc, lddt, lddx, lddb, lddc, ldddt, p.chunk, p.chunks, ws + p.state0, ws + p.adj, ws + p.log,
                     p.parts == 1 ? nullptr : ws + p.db, p.parts == 1 ? nullptr : ws + p.dc, ws + p.part, ws + p.kept, nullptr};
    s = device_error_word(&a.err, why);
    if (s != IDA_OK) return fail_with(s, why);
    if (!p.tc) return dtype == IDA_F32 ? launch_bwd_m<float>(a, st) : launch_bwd_m<__nv_bfloat16>(a, st);
    s = launch_bwd_tc_states(a, st);
    if (s == IDA_OK) s = launch_bwd_carry(a, st);
    if (s == IDA_OK) s = launch_bwd_tc(a, p.parts, st);
    return s == IDA_OK ? launch_bwd_sums<__nv_bfloat16>(a, p.parts, 4, st) : s;
}

}  // extern "C"
