// ida_ssm_scan.cu -- the selective scan position by position on the CUDA cores (fp32 inputs,
// and the segment states it is split by), and the entry point.
//
// A warp owns 32 columns of a head's state: lane l holds the M / 4 rows of quarter l % 4 of the
// four columns 4 (l / 4) .., in registers, as pairs of rows for the packed fp32x2 instructions,
// so that b and c come from shared memory as 16-byte broadcasts and only y is summed across
// lanes (three shuffles a position, after which lane l holds column l).  Per position that is
// three packed operations for two state elements; the fp32 rate of the CUDA cores bounds it.
// Positions go in tiles of SEQ_T: the next tile's raw rows are copied asynchronously while the
// present one's, converted to fp32 (b times its step size), are walked.
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

// Shared memory of a CTA of `cols` columns.
template <typename E, int MT>
struct SeqSmem {
    static constexpr int QS = MT + 4;      // floats of a quarter row: the four quarters on their own banks
    static constexpr int MS = 4 * QS;      // floats of a row of b or c
    __host__ __device__ static size_t raw_bytes(int cols) { return (size_t)SEQ_T * (8 * MT + cols) * sizeof(E); }
    __host__ __device__ static size_t bytes(int cols) {
        return raw_bytes(cols) + (size_t)SEQ_T * (2 * MS + cols) * sizeof(float) + 4 * SEQ_T * sizeof(float);
    }
};

// MT: state rows per lane (M <= 4 MT).  STATE: only the segment's last state from zero.
template <typename E, int MT, bool STATE>
__global__ void __launch_bounds__(128) scan_seq_kernel(ScanArgs a) {
    using V = Vec16<E>;
    using S = SeqSmem<E, MT>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int M = a.M, d = a.d, H = a.H, N = a.N, rep = H / a.G;
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cols = nt;
    const int slices = (d + cols - 1) / cols, nseg = STATE ? a.state_segs : a.segs;
    int id = blockIdx.x;
    const int seg = id % nseg;
    id /= nseg;
    const int j0 = id % slices * cols;
    const int unit = id / slices, b = unit / H, h = unit % H, g = h / rep;
    E *raw = reinterpret_cast<E *>(smem);  // [T][b 4 MT | c 4 MT | x cols]
    float *fb = reinterpret_cast<float *>(smem + S::raw_bytes(cols)), *fc = fb + SEQ_T * S::MS;
    float *fx = fc + SEQ_T * S::MS, *fad = fx + SEQ_T * cols;  // fad: decays and step sizes, two tiles' in turn
    constexpr int RS = 8 * MT;  // raw row: b, c, then x
    const int rs = RS + cols;
    const int t_begin = seg * a.seg, t_end = min(N, t_begin + a.seg);
    const E *gb = static_cast<const E *>(a.b) + (size_t)b * N * a.ldb + g * M;
    const E *gc = static_cast<const E *>(a.c) + (size_t)b * N * a.ldc + g * M;
    const E *gx = static_cast<const E *>(a.x) + (size_t)b * N * a.ldx + (size_t)h * d + j0;
    const E *gdt = static_cast<const E *>(a.dt) + (size_t)b * N * a.lddt + h;
    const float rate = expf(a.a_log[h]), dt_bias = a.dt_bias[h], skip = STATE ? 0.f : a.D[h];

    const auto fetch = [&](int t0) {
        const int vpr = rs / V::n;
        for (int i = tid; i < SEQ_T * vpr; i += nt) {
            const int t = i / vpr, e = i % vpr * V::n, p = t0 + t;
            const E *src = gx;
            bool ok = p < t_end;
            if (e < 4 * MT) {
                ok = ok && e < M;
                src = gb + (size_t)p * a.ldb + e;
            } else if (e < RS) {
                ok = ok && !STATE && e - 4 * MT < M;
                src = gc + (size_t)p * a.ldc + (e - 4 * MT);
            } else {
                ok = ok && j0 + e - RS < d;
                src = gx + (size_t)p * a.ldx + (e - RS);
            }
            cp_async16(raw + t * rs + e, ok ? src : gx, ok);
        }
        cp_async_commit();
    };

    const int km = lane & 3, jl = warp * 32 + (lane >> 2) * 4;  // my quarter of rows, my first column
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
                    const float4 u = __ldg(reinterpret_cast<const float4 *>(p + (size_t)m * d + j0 + jl));
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(p + (size_t)(m + 1) * d + j0 + jl));
                    X[i][0] = ssm_fma(X[i][0], ff, ssm_pack(u.x, v.x));
                    X[i][1] = ssm_fma(X[i][1], ff, ssm_pack(u.y, v.y));
                    X[i][2] = ssm_fma(X[i][2], ff, ssm_pack(u.z, v.z));
                    X[i][3] = ssm_fma(X[i][3], ff, ssm_pack(u.w, v.w));
                }
            }
        }
    }
    double log_sum = 0.0;  // thread 0

    fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += SEQ_T) {
        float *fa = fad + (((t0 - t_begin) / SEQ_T) & 1) * 2 * SEQ_T, *fd = fa + SEQ_T;
        if (warp == 0) {
            float la = 0.f;
            if (lane < SEQ_T) {
                const int p = t0 + lane;
                float delta = 0.f;  // behind the end nothing decays or is added
                if (p < t_end) delta = softplus(to_float(gdt[(size_t)p * a.lddt]) + dt_bias);
                la = -rate * delta;
                fd[lane] = delta;
                fa[lane] = expf(la);
            }
            if (STATE) {
                la = warp_sum(la);
                log_sum += la;
            }
        }
        cp_async_wait_all();
        __syncthreads();  // raw rows and step sizes are there, and the walk of the last tile is done
        for (int i = tid; i < SEQ_T * (rs / V::n); i += nt) {
            const int t = i / (rs / V::n), e = i % (rs / V::n) * V::n;
            float v[V::n];
            V::unpack(*reinterpret_cast<const uint4 *>(raw + t * rs + e), v);
            float *dst;
            if (e < RS) {
                const int m = e < 4 * MT ? e : e - 4 * MT;
                dst = (e < 4 * MT ? fb : fc) + t * S::MS;
                const float f = e < 4 * MT ? fd[t] : 1.f;
#pragma unroll
                for (int k = 0; k < V::n; ++k) {
                    const int mk = m + k;
                    dst[mk / MT * S::QS + mk % MT] = v[k] * f;
                }
            } else {
                dst = fx + t * cols + (e - RS);
#pragma unroll
                for (int k = 0; k < V::n; ++k) dst[k] = v[k];
            }
        }
        __syncthreads();
        if (t0 + SEQ_T < t_end) fetch(t0 + SEQ_T);
        const int len = min(SEQ_T, t_end - t0);
        for (int t = 0; t < len; ++t) {
            const float4 x4 = *reinterpret_cast<const float4 *>(fx + t * cols + jl);
            const float av = fa[t];
            const ssm_f2 aa = ssm_pack(av, av);
            const ssm_f2 xx[4] = {ssm_pack(x4.x, x4.x), ssm_pack(x4.y, x4.y), ssm_pack(x4.z, x4.z), ssm_pack(x4.w, x4.w)};
            const float *pb = fb + t * S::MS + km * S::QS, *pc = fc + t * S::MS + km * S::QS;
            ssm_f2 acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int i = 0; i < MT / 2; i += 2) {
                const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(pb + 2 * i);
                ulonglong2 c2;
                if (!STATE) c2 = *reinterpret_cast<const ulonglong2 *>(pc + 2 * i);
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
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    ssm_unpack(acc[j], lo, hi);
                    y[j] = lo + hi;
                }
                // sum over the four quarters: lane l ends with column l of the warp
                const bool up = (lane & 2) != 0, odd = (lane & 1) != 0;
                const float k0 = (up ? y[2] : y[0]) + __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 2);
                const float k1 = (up ? y[3] : y[1]) + __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 2);
                const float o = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
                const int col = warp * 32 + lane;
                if (j0 + col < d)
                    from_float(static_cast<E *>(a.y) + (((size_t)b * N + t0 + t) * H + h) * d + j0 + col,
                               fmaf(skip, fx[t * cols + col], o));
            }
        }
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
    if (STATE && tid == 0 && j0 == 0) a.seg_log[(size_t)unit * a.segs + seg] = (float)log_sum;
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

template <typename E, int MT>
static ida_status launch_seq(const ScanArgs &a, cudaStream_t st) {
    const int cols = seq_cols(a.d), slices = (a.d + cols - 1) / cols;
    const size_t smem = SeqSmem<E, MT>::bytes(cols);
    const long long units = (long long)a.B * a.H * slices;
    if (units * a.segs > 0x7FFFFFFFLL) return fail_with(IDA_ERR_UNSUPPORTED, "too many rows and heads");
    cudaError_t e = cudaFuncSetAttribute(scan_seq_kernel<E, MT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(scan_seq_kernel<E, MT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail_with(IDA_ERR_CUDA, cudaGetErrorString(e));
    if (a.state_segs > 0) {
        scan_seq_kernel<E, MT, true><<<(unsigned)(units * a.state_segs), cols, smem, st>>>(a);
        const ida_status s = launched("ssm segment states");
        if (s != IDA_OK) return s;
    }
    scan_seq_kernel<E, MT, false><<<(unsigned)(units * a.segs), cols, smem, st>>>(a);
    return launched("ssm scan");
}

template <typename E>
static ida_status launch_seq_m(const ScanArgs &a, cudaStream_t st) {
    if (a.M <= 16) return launch_seq<E, 4>(a, st);
    if (a.M <= 32) return launch_seq<E, 8>(a, st);
    if (a.M <= 64) return launch_seq<E, 16>(a, st);
    return launch_seq<E, 32>(a, st);
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
    if (overlap(state_in, state_bytes, final_state, state_bytes))
        return fail_with(IDA_ERR_ARG, "state_in and final_state must not overlap");
    if (N > 0) {
        const void *ptrs[] = {x, b, c, a_log, dt_bias, D, y};
        for (const void *p : ptrs) {
            if (!p) return fail_with(IDA_ERR_ARG, "null input or output pointer");
            if (misaligned16(p)) return fail_with(IDA_ERR_ARG, "pointers must be 16-byte aligned");
        }
        if (!dt || (reinterpret_cast<uintptr_t>(dt) % (dtype == IDA_F32 ? 4 : 2)))
            return fail_with(IDA_ERR_ARG, "dt must be an aligned pointer");
    }
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
        a.seg_state = static_cast<float *>(workspace);
        a.seg_log = a.seg_state + (size_t)B * H * a.segs * a.fine * M * d;
    } else {
        a.seg = (N + 127) / 128 * 128;
        a.segs = a.fine = 1;
    }
    // the tensor-core kernel takes a final state from segment states, the other one from its own
    a.state_segs = chunked && final_state ? a.segs * a.fine : (a.segs - 1) * a.fine;
    return chunked ? launch_ssm_chunk(a, st) : launch_seq_m<float>(a, st);
}

}  // extern "C"
