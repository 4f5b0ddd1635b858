// ida_ssm_scan.cu -- the selective scan position by position on the CUDA cores (fp32 inputs,
// and the segment states it is split by), and the entry point.
//
// A warp owns 32 columns of a head's state: lane l holds the M / 4 rows of quarter l % 4 of the
// four columns 4 (l / 4) .., in registers, as pairs of rows for the packed fp32x2 instructions,
// so that b and c come from shared memory as 16-byte broadcasts and only y is summed across
// lanes (three shuffles a position, after which lane l holds column l).  Per position that is
// three packed operations for two state elements; the fp32 rate of the CUDA cores bounds it.
// Positions go in tiles of SEQ_T, in two buffers: four helper warps read the next tile's rows, form
// its step sizes and lay it out (b times its step size) while the others walk the present one.
// (Converted by the walking warps themselves, 251 positions of 2 heads of 32 x 16 took 54 us, most
// of it the conversion.)
//
// Few (row, head) units do not fill the SMs.  With a workspace a sequence is cut into segments:
// a first launch leaves each segment's last state from zero, and the second starts every segment
// from the decayed sum of the states before it.
#include "ida_ssm.cuh"

namespace ida {

ida_status device_error_word(unsigned **err, std::string &why);
ida_status launch_ssm_chunk(const ScanArgs &a, cudaStream_t st);
void ssm_chunk_segments(int B, int H, int N, int d, int M, int num_sms, int &seg, int &segs, int &fine);

constexpr int SEQ_T = 16;  // positions per tile

constexpr int SEQ_HELP = 128;  // helper threads

// Floats of a tile of `cols` columns: rows of b and c (four quarters on their own banks), of x, decays.
template <int MT>
struct SeqTile {
    static constexpr int QS = MT + 4, MS = 4 * QS;
    __host__ __device__ static int floats(int cols) { return SEQ_T * (2 * MS + cols + 1); }
};

// MT: state rows per lane (M <= 4 MT).  STATE: only the segment's last state from zero.
template <int MT, bool STATE>
__global__ void __launch_bounds__(128 + SEQ_HELP) scan_seq_kernel(ScanArgs a) {
    using L = SeqTile<MT>;
    extern __shared__ __align__(16) float sm[];
    if (STATE)
        dependent_launch();
    else
        dependent_wait();
    const int M = a.M, d = a.d, H = a.H, N = a.N, rep = H / a.G;
    const int cols = blockDim.x - SEQ_HELP, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = (d + cols - 1) / cols, nseg = STATE ? a.state_segs : a.segs;
    int id = blockIdx.x;
    const int seg = id % nseg;
    id /= nseg;
    const int j0 = id % slices * cols;
    const int unit = id / slices, b = unit / H, h = unit % H, g = h / rep;
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg);
    const int tile = L::floats(cols);  // [T][MS] b, [T][MS] c, [T][cols] x, [T] decays

    if (tid >= cols) {
        // helpers: a thread keeps its 16-byte column of [b | c | x] and walks the tile's rows
        const int ht = tid - cols, nb = M / 4, nx = min(cols, d - j0) / 4, vpr = (STATE ? nb : 2 * nb) + nx;
        const float *dt = static_cast<const float *>(a.dt) + (size_t)b * N * a.lddt + h;
        const float rate = scan_rate(a.a_log[h]), dt_bias = a.dt_bias[h];
        const float *src = nullptr;
        long long ld = 0;
        int at = 0, rs = 0;  // the column's place in a tile, and its row stride there
        bool is_b = false;
        const int step = vpr < SEQ_HELP ? SEQ_HELP / vpr : 1;  // rows the helpers take at a time
        double log_sum = 0.0;
        const auto column = [&](int v) {
            if (v < nb) {
                is_b = true;
                src = static_cast<const float *>(a.b) + (size_t)b * N * a.ldb + g * M + 4 * v;
                ld = a.ldb;
                at = 4 * v / MT * L::QS + 4 * v % MT;
                rs = L::MS;
            } else if (!STATE && v < 2 * nb) {
                is_b = false;
                v -= nb;
                src = static_cast<const float *>(a.c) + (size_t)b * N * a.ldc + g * M + 4 * v;
                ld = a.ldc;
                at = SEQ_T * L::MS + 4 * v / MT * L::QS + 4 * v % MT;
                rs = L::MS;
            } else {
                is_b = false;
                v -= STATE ? nb : 2 * nb;
                src = static_cast<const float *>(a.x) + (size_t)b * N * a.ldx + (size_t)h * d + j0 + 4 * v;
                ld = a.ldx;
                at = 2 * SEQ_T * L::MS + 4 * v;
                rs = cols;
            }
        };
        const auto fill = [&](int t0, float *buf) {
            for (int v = ht % (vpr < SEQ_HELP ? vpr : SEQ_HELP); v < vpr; v += SEQ_HELP) {
                const int r0 = vpr < SEQ_HELP ? ht / vpr : 0;
                if (r0 >= step) break;  // spare helpers
                column(v);
#pragma unroll 4
                for (int t = r0; t < SEQ_T; t += step) {
                    const int p = t0 + t;
                    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p < t_end) {
                        u = __ldg(reinterpret_cast<const float4 *>(src + (size_t)p * ld));
                        if (is_b) {
                            const float f = softplus(__ldg(dt + (size_t)p * a.lddt) + dt_bias);
                            u = make_float4(f * u.x, f * u.y, f * u.z, f * u.w);
                        }
                    }
                    *reinterpret_cast<float4 *>(buf + at + t * rs) = u;
                }
            }
            if (ht < 32) {
                float la = 0.f;
                if (ht < SEQ_T && t0 + ht < t_end) la = -rate * softplus(dt[(size_t)(t0 + ht) * a.lddt] + dt_bias);
                if (ht < SEQ_T) buf[SEQ_T * (2 * L::MS + cols) + ht] = expf(la);  // behind the end nothing decays or is added
                if (STATE) log_sum += warp_sum(la);
            }
        };
        // columns that no vector fills: rows of b and c behind M, columns of x behind d
        for (int i = ht; i < 2 * tile; i += SEQ_HELP) sm[i] = 0.f;
        named_sync(1, SEQ_HELP);
        fill(t_begin, sm);
        __syncthreads();
        int k = 1;
        for (int t0 = t_begin; t0 < t_end; t0 += SEQ_T, ++k) {
            if (t0 + SEQ_T < t_end) fill(t0 + SEQ_T, sm + (k & 1) * tile);
            __syncthreads();
        }
        if (STATE && ht == 0 && j0 == 0) a.seg_log[(size_t)unit * a.segs + seg] = (float)log_sum;
        return;
    }

    const int km = lane & 3, jl = warp * 32 + (lane >> 2) * 4;  // my quarter of rows, my first column
    const float skip = STATE ? 0.f : a.D[h];
    ssm_f2 X[MT / 2][4];
#pragma unroll
    for (int i = 0; i < MT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) X[i][j] = 0ull;
    if (!STATE) {
        // the state before the segment: the given one and the segments before, decayed
        const bool mine = j0 + jl < d;
        const float *in = a.state_in ? a.state_in + (size_t)unit * M * d : nullptr;
        for (int s = -1; s < seg; ++s) {
            const float *p = s < 0 ? in : a.seg_state + ((size_t)unit * a.segs + s) * M * d;
            const float f = s < 0 ? 0.f : expf(a.seg_log[(size_t)unit * a.segs + s]);
            const ssm_f2 ff = ssm_pack(f, f);
            if (!p || !mine) continue;
#pragma unroll
            for (int i = 0; i < MT / 2; ++i) {
                const int m = km * MT + 2 * i;
                if (m < M) {
                    const float4 u = __ldcg(reinterpret_cast<const float4 *>(p + (size_t)m * d + j0 + jl));
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + (size_t)(m + 1) * d + j0 + jl));
                    X[i][0] = ssm_fma(X[i][0], ff, ssm_pack(u.x, v.x));
                    X[i][1] = ssm_fma(X[i][1], ff, ssm_pack(u.y, v.y));
                    X[i][2] = ssm_fma(X[i][2], ff, ssm_pack(u.z, v.z));
                    X[i][3] = ssm_fma(X[i][3], ff, ssm_pack(u.w, v.w));
                }
            }
        }
    }
    const int col = warp * 32 + lane;  // the column whose y I hold after the sum over quarters
    float *y = static_cast<float *>(a.y) + (((size_t)b * N + t_begin) * H + h) * d + j0 + col;
    const size_t ys = (size_t)H * d;
    const bool has = j0 + col < d;
    __syncthreads();
    int k = 0;
    for (int t0 = t_begin; t0 < t_end; t0 += SEQ_T, ++k, y += SEQ_T * ys) {
        const float *fb = sm + (k & 1) * tile + km * L::QS, *fc = fb + SEQ_T * L::MS;
        const float *fx = sm + (k & 1) * tile + 2 * SEQ_T * L::MS, *fa = fx + SEQ_T * cols;
        const int left = t_end - t0;
#pragma unroll(MT <= 8 ? 4 : 1)
        for (int t = 0; t < SEQ_T; ++t) {  // positions behind the end change nothing
            const float4 x4 = *reinterpret_cast<const float4 *>(fx + t * cols + jl);
            const float av = fa[t];
            const ssm_f2 aa = ssm_pack(av, av);
            const ssm_f2 xx[4] = {ssm_pack(x4.x, x4.x), ssm_pack(x4.y, x4.y), ssm_pack(x4.z, x4.z), ssm_pack(x4.w, x4.w)};
            ssm_f2 acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int i = 0; i < MT / 2; i += 2) {
                const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(fb + t * L::MS + 2 * i);
                ulonglong2 c2;
                if (!STATE) c2 = *reinterpret_cast<const ulonglong2 *>(fc + t * L::MS + 2 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    X[i][j] = ssm_fma(b2.x, xx[j], ssm_mul(aa, X[i][j]));
                    X[i + 1][j] = ssm_fma(b2.y, xx[j], ssm_mul(aa, X[i + 1][j]));
                    if (!STATE) {
                        acc[j] = ssm_fma(c2.x, X[i][j], acc[j]);
                        acc[j] = ssm_fma(c2.y, X[i + 1][j], acc[j]);
                    }
                }
            }
            if (!STATE) {
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    ssm_unpack(acc[j], lo, hi);
                    o[j] = lo + hi;
                }
                // sum over the four quarters: lane l ends with column l of the warp
                const bool up = (lane & 2) != 0, odd = (lane & 1) != 0;
                const float k0 = (up ? o[2] : o[0]) + __shfl_xor_sync(0xffffffffu, up ? o[0] : o[2], 2);
                const float k1 = (up ? o[3] : o[1]) + __shfl_xor_sync(0xffffffffu, up ? o[1] : o[3], 2);
                const float v = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
                if (has && t < left) y[t * ys] = fmaf(skip, fx[t * cols + col], v);
            }
        }
        __syncthreads();
    }
    float *out = STATE ? a.seg_state + ((size_t)unit * a.segs + seg) * M * d
                       : (a.final_state && seg == a.segs - 1 ? a.final_state + (size_t)unit * M * d : nullptr);
    if (out && j0 + jl < d)
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
            const int m = km * MT + 2 * i;
            if (m < M) {
                float u[4], v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ssm_unpack(X[i][j], u[j], v[j]);
                *reinterpret_cast<float4 *>(out + (size_t)m * d + j0 + jl) = make_float4(u[0], u[1], u[2], u[3]);
                *reinterpret_cast<float4 *>(out + (size_t)(m + 1) * d + j0 + jl) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
}

static int seq_cols(int d) { return d >= 128 ? 128 : (d + 31) / 32 * 32; }

// Segments of the CUDA-core scan: enough for two CTAs per SM, of 64 positions at least.  The
// state launch repeats two thirds of the work of all segments but the last, so a split that
// would not at least double the CTAs is not made.
static void seq_segments(int B, int H, int N, int d, int num_sms, int &seg, int &segs) {
    const int cols = seq_cols(d);
    const long long ctas = (long long)B * H * ((d + cols - 1) / cols);
    long long want = ctas > 0 ? 2LL * num_sms / ctas : 1;
    want = want < 3 ? 1 : want;
    if (want > N / 64) want = N / 64;
    if (want < 1) want = 1;
    seg = (int)(((N + want - 1) / want + SEQ_T - 1) / SEQ_T * SEQ_T);
    if (seg < SEQ_T) seg = SEQ_T;
    segs = (N + seg - 1) / seg;
}

// The split of a call and the bytes of its segment states.
static size_t scan_plan(int B, int H, int N, int d, int M, bool chunked, int num_sms, int &seg, int &segs, int &fine) {
    fine = 1;
    if (chunked)
        ssm_chunk_segments(B, H, N, d, M, num_sms, seg, segs, fine);
    else
        seq_segments(B, H, N, d, num_sms, seg, segs);
    return segs < 2 ? 0 : (size_t)B * H * segs * fine * ((size_t)M * d + 4) * sizeof(float);
}

template <int MT>
static ida_status launch_seq(const ScanArgs &a, cudaStream_t st) {
    const int cols = seq_cols(a.d), slices = (a.d + cols - 1) / cols;
    const size_t smem = 2 * (size_t)SeqTile<MT>::floats(cols) * sizeof(float);
    const long long units = (long long)a.B * a.H * slices;
    if (units * a.segs > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows and heads");
    cudaError_t e = allow_smem(scan_seq_kernel<MT, false>, smem);
    if (e == cudaSuccess) e = allow_smem(scan_seq_kernel<MT, true>, smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    if (a.state_segs > 0) {
        scan_seq_kernel<MT, true><<<(unsigned)(units * a.state_segs), cols + SEQ_HELP, smem, st>>>(a);
        const ida_status s = launched("ssm segment states");
        if (s != IDA_OK) return s;
        e = launch_dependent(scan_seq_kernel<MT, false>, dim3((unsigned)(units * a.segs)), dim3(cols + SEQ_HELP), smem, st, a);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, std::string("ssm scan launch: ") + cudaGetErrorString(e));
    }
    scan_seq_kernel<MT, false><<<(unsigned)(units * a.segs), cols + SEQ_HELP, smem, st>>>(a);
    return launched("ssm scan");
}

static ida_status launch_seq_m(const ScanArgs &a, cudaStream_t st) {
    if (a.M <= 16) return launch_seq<4>(a, st);
    if (a.M <= 32) return launch_seq<8>(a, st);
    if (a.M <= 64) return launch_seq<16>(a, st);
    return launch_seq<32>(a, st);
}

ida_status check_scan(int B, int H, int N, int d, int G, int M, long long ldx, long long ldb, long long ldc, long long lddt,
                      int dtype) {
    if (B < 0 || H < 0 || N < 0) return fail_with(IDA_ERR_ARG, "B, H and N must be >= 0");
    ida_status s = check_ssm(H, d, G, M, dtype);
    if (s != IDA_OK) return s;
    if (ldx < (long long)H * d || ldb < (long long)G * M || ldc < (long long)G * M || lddt < H)
        return fail_with(IDA_ERR_ARG, "a row stride is below its row");
    if ((ldx % 8) || (ldb % 8) || (ldc % 8)) return fail_with(IDA_ERR_UNSUPPORTED, "the row strides of x, b and c must be multiples of 8");
    const long long top = 1LL << 32;
    if (ldx > top || ldb > top || ldc > top || lddt > top) return fail_with(IDA_ERR_UNSUPPORTED, "a row stride above 2^32");
    if ((long long)B * H > (1LL << 24)) return fail_with(IDA_ERR_UNSUPPORTED, "B*H above 2^24");
    if ((long long)B * N > (1LL << 28)) return fail_with(IDA_ERR_UNSUPPORTED, "B*N above 2^28");
    return IDA_OK;
}

}  // namespace ida

extern "C" {

size_t ida_ssm_scan_workspace_bytes(int B, int H, int N, int d, int G, int M, int dtype) {
    using namespace ida;
    if (check_scan(B, H, N, d, G, M, (long long)H * d, (long long)G * M, (long long)G * M, H, dtype) != IDA_OK) return 0;
    if ((long long)B * H * N == 0) return 0;
    int dev = 0, num_sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    int seg, segs, fine;
    return scan_plan(B, H, N, d, M, dtype == IDA_BF16, num_sms, seg, segs, fine);
}

ida_status ida_ssm_scan(const void *x, const void *b, const void *c, const void *dt, const float *a_log,
                        const float *dt_bias, const float *D, const float *state_in, void *y, float *final_state,
                        int B, int H, int N, int d, int G, int M, long long ldx, long long ldb, long long ldc, long long lddt,
                        int dtype, void *workspace, size_t workspace_bytes, ida_stream_t stream) {
    using namespace ida;
    ida_status s = check_scan(B, H, N, d, G, M, ldx, ldb, ldc, lddt, dtype);
    if (s != IDA_OK) return s;
    if ((long long)B * H == 0 || (N == 0 && !final_state)) return IDA_OK;
    const size_t state_bytes = (size_t)B * H * M * d * sizeof(float);
    if (misaligned16(state_in) || misaligned16(final_state) || misaligned16(workspace))
        return fail_with(IDA_ERR_ARG, "state_in, final_state and workspace must be 16-byte aligned");
    if (N > 0) {
        const void *ptrs[] = {x, b, c, a_log, dt_bias, D, y};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        if (!dt || (reinterpret_cast<uintptr_t>(dt) % (dtype == IDA_F32 ? 4 : 2)))
            return fail_with(IDA_ERR_ARG, "dt must be an aligned pointer");
    }
    const long long rows = (long long)B * N, w = (long long)H * d, bc = (long long)G * M;
    const size_t par = N > 0 ? (size_t)H * 4 : 0;
    const auto refuse_overlaps = [&](size_t workspace_used) {
        const Rows outs[] = {rows_of("y", y, w, w, rows, dtype), dense("final_state", final_state, state_bytes),
                             dense("workspace", workspace, workspace_used)};
        const Rows ins[] = {rows_of("x", x, ldx, w, rows, dtype), rows_of("b", b, ldb, bc, rows, dtype), rows_of("c", c, ldc, bc, rows, dtype),
                            rows_of("dt", dt, lddt, H, rows, dtype), dense("a_log", a_log, par), dense("dt_bias", dt_bias, par),
                            dense("D", D, par), dense("state_in", state_in, state_bytes)};
        return check_overlaps(outs, ins);
    };
    s = refuse_overlaps(0);
    if (s != IDA_OK) return s;
    int num_sms = 0;
    std::string why;
    s = device_ready(&num_sms, why);
    if (s != IDA_OK) return fail_with(s, why);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {  // no positions: the state is handed on
        cudaError_t e = state_in ? cudaMemcpyAsync(final_state, state_in, state_bytes, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(final_state, 0, state_bytes, st);
        return e == cudaSuccess ? IDA_OK : fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    }
    ScanArgs a = {x, b, c, dt, a_log, dt_bias, D, state_in, y, final_state, B, H, N, d, G, M, ldx, ldb, ldc, lddt,
                  0, 0, 1, 0, nullptr, nullptr, nullptr};
    s = device_error_word(&a.err, why);
    if (s != IDA_OK) return fail_with(s, why);
    const bool chunked = dtype == IDA_BF16;
    const size_t need = scan_plan(B, H, N, d, M, chunked, num_sms, a.seg, a.segs, a.fine);
    if (need > 0 && workspace && workspace_bytes >= need) {
        s = refuse_overlaps(need);
        if (s != IDA_OK) return s;
        a.seg_state = static_cast<float *>(workspace);
        a.seg_log = a.seg_state + (size_t)B * H * a.segs * a.fine * M * d;
    } else {
        a.seg = (N + 127) / 128 * 128;
        a.segs = a.fine = 1;
    }
    // the tensor-core kernel takes a final state from segment states, the other one from its own
    a.state_segs = chunked && final_state ? a.segs * a.fine : (a.segs - 1) * a.fine;
    return chunked ? launch_ssm_chunk(a, st) : launch_seq_m(a, st);
}

}  // extern "C"
