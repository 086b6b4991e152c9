// The gated linear recurrence and its gradients (fi_scan_*).
//
// With d_t = 1 - sigmoid(z_t) and b_t = e(d_t) x_t a position is the map
// s -> s - d_t s + b_t, affine in the state, and so is a run of positions:
// s -> A s + S.  The length is cut into chunks; the maps of all chunks are
// formed at once, the states at the chunks' ends follow one from the other,
// and every chunk then runs from its own start state.  The gradients are the
// same recurrence from the end: D_t = dy_t + c, c <- D_t - d_t D_t.
//
// The state is updated as s - d s, never as a s with a = 1 - d rounded to
// fp32: for decays near one (a memory of thousands of positions) the rounding
// of a alone is a relative error of 2^-25 / d in the memory's length.
#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kScanChunk = 256;   // positions per chunk, and per state that is kept for the backward pass
constexpr int kScanSub = 16;      // states held in registers at a time by the backward pass

struct ScanArgs {
    const void *x, *gate, *dy;
    void *y, *dx, *dgate;
    const float *bias, *state, *dfinal;
    float *final, *dstate;
    const int32_t *lengths;
    float *saved;              // [chunks][R] state after each chunk
    float *mul, *add;          // [chunks][R] maps of the chunks
    float *pbias;              // [chunks][R] partial sums of the bias gradient
    int64_t T;
    int64_t ldx, ldg, ldy, lddy, lddx, lddg;
    int B, D;
    int chunks;
};

__device__ __forceinline__ float sigmoid_neg(float z) {   // 1 - sigmoid(z) = 1 / (1 + e^z)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * 1.44269504088896f));
}

template <int IN>
__device__ __forceinline__ float input_factor(float d) {
    if (IN == FI_SCAN_PLAIN) return 1.f;
    if (IN == FI_SCAN_CONVEX) return d;
    return __builtin_amdgcn_sqrtf(d * (2.f - d));
}

// ds/dz of one position: the decay's part d(1-d) s_{t-1} and the input factor's.
template <int IN>
__device__ __forceinline__ float gate_slope(float d, float x, float before) {
    const float a = 1.f - d;
    if (IN == FI_SCAN_PLAIN) return a * d * before;
    if (IN == FI_SCAN_CONVEX) return a * d * (before - x);
    return a * (d * before - a * __builtin_amdgcn_sqrtf(d * __builtin_amdgcn_rcpf(2.f - d)) * x);
}

struct Column {                 // one (b, c) column of one chunk
    int64_t t0, t1, end;        // the chunk's positions, and where the row's own positions end
    int r, b, c;
    float bias;
};

__device__ __forceinline__ bool column(const ScanArgs &p, Column &k) {
    k.r = blockIdx.x * blockDim.x + threadIdx.x;
    if (k.r >= p.B * p.D) return false;
    k.b = k.r / p.D;
    k.c = k.r - k.b * p.D;
    k.t0 = (int64_t)blockIdx.y * kScanChunk;
    k.t1 = k.t0 + kScanChunk < p.T ? k.t0 + kScanChunk : p.T;
    int64_t len = p.T;
    if (p.lengths) {
        const int64_t n = p.lengths[k.b];
        len = n < 0 ? 0 : n < p.T ? n : p.T;
    }
    k.end = len < k.t1 ? (len < k.t0 ? k.t0 : len) : k.t1;
    k.bias = p.bias ? p.bias[k.c] : 0.f;
    return true;
}

template <typename V>
__device__ __forceinline__ float at(const void *p, int64_t row, int64_t ld, int c) {
    return (float)static_cast<const V *>(p)[row * ld + c];
}

// The map of one chunk of one column.
template <typename V, int IN>
__global__ void __launch_bounds__(64) k_scan_map(ScanArgs p) {
    Column k;
    if (!column(p, k)) return;
    float A = 1.f, S = 0.f;
    for (int64_t t = k.t0; t < k.end; ++t) {
        const int64_t row = t * p.B + k.b;
        const float d = sigmoid_neg(at<V>(p.gate, row, p.ldg, k.c) + k.bias);
        const float x = at<V>(p.x, row, p.ldx, k.c);
        S = S + fmaf(-d, S, input_factor<IN>(d) * x);
        A = fmaf(-d, A, A);
    }
    const size_t i = (size_t)blockIdx.y * (p.B * (size_t)p.D) + k.r;
    p.mul[i] = A;
    p.add[i] = S;
}

// States at the chunks' ends, one column per thread.
__global__ void __launch_bounds__(64) k_scan_carry(ScanArgs p, float *ends) {
    const size_t R = p.B * (size_t)p.D, r = blockIdx.x * (size_t)64 + threadIdx.x;
    if (r >= R) return;
    float s = p.state ? p.state[r] : 0.f;
    for (int j = 0; j < p.chunks; ++j) {
        const float A = p.mul[j * R + r], S = p.add[j * R + r];
        if (j == 0) p.mul[r] = s;     // final may be state: the last chunk writes it while the first one runs
        s = fmaf(A, s, S);
        ends[j * R + r] = s;
    }
}

template <typename V, int IN>
__global__ void __launch_bounds__(64) k_scan_apply(ScanArgs p, const float *ends) {
    Column k;
    if (!column(p, k)) return;
    const size_t R = p.B * (size_t)p.D;
    float s = blockIdx.y ? ends[(blockIdx.y - 1) * R + k.r]
                         : p.chunks > 1 ? p.mul[k.r] : p.state ? p.state[k.r] : 0.f;
    V *y = static_cast<V *>(p.y);
    for (int64_t t = k.t0; t < k.end; ++t) {
        const int64_t row = t * p.B + k.b;
        const float d = sigmoid_neg(at<V>(p.gate, row, p.ldg, k.c) + k.bias);
        const float x = at<V>(p.x, row, p.ldx, k.c);
        s = s + fmaf(-d, s, input_factor<IN>(d) * x);
        y[row * p.ldy + k.c] = (V)s;
    }
    for (int64_t t = k.end; t < k.t1; ++t) y[(t * p.B + k.b) * p.ldy + k.c] = (V)0.f;
    if (p.saved && p.chunks == 1) p.saved[k.r] = s;
    if (p.final && (int)blockIdx.y == p.chunks - 1) p.final[k.r] = s;
}

// The backward maps: c at a chunk's end -> c before its start, c = (1 - d) D.
template <typename V>
__global__ void __launch_bounds__(64) k_scan_bmap(ScanArgs p) {
    Column k;
    if (!column(p, k)) return;
    float A = 1.f, S = 0.f;
    for (int64_t t = k.end - 1; t >= k.t0; --t) {
        const int64_t row = t * p.B + k.b;
        const float d = sigmoid_neg(at<V>(p.gate, row, p.ldg, k.c) + k.bias);
        const float g = at<V>(p.dy, row, p.lddy, k.c) + S;
        S = fmaf(-d, g, g);
        A = fmaf(-d, A, A);
    }
    const size_t i = (size_t)blockIdx.y * (p.B * (size_t)p.D) + k.r;
    p.mul[i] = A;
    p.add[i] = S;
}

// c arriving at each chunk's end (into mul), one column per thread, from the last chunk.
__global__ void __launch_bounds__(64) k_scan_bcarry(ScanArgs p) {
    const size_t R = p.B * (size_t)p.D, r = blockIdx.x * (size_t)64 + threadIdx.x;
    if (r >= R) return;
    float c = p.dfinal ? p.dfinal[r] : 0.f;
    for (int j = p.chunks - 1; j >= 0; --j) {
        const float A = p.mul[j * R + r], S = p.add[j * R + r];
        p.mul[j * R + r] = c;
        c = fmaf(A, c, S);
    }
}

template <typename V, int IN>
__global__ void __launch_bounds__(64) k_scan_bapply(ScanArgs p) {
    Column k;
    if (!column(p, k)) return;
    const size_t R = p.B * (size_t)p.D;
    const int j = blockIdx.y;
    V *dx = static_cast<V *>(p.dx), *dg = static_cast<V *>(p.dgate);
    for (int64_t t = k.end; t < k.t1; ++t) {
        dx[(t * p.B + k.b) * p.lddx + k.c] = (V)0.f;
        dg[(t * p.B + k.b) * p.lddg + k.c] = (V)0.f;
    }
    // states before each sub-run of kScanSub positions
    float start[kScanChunk / kScanSub];
    float s = j ? p.saved[(j - 1) * R + k.r] : p.state ? p.state[k.r] : 0.f;
#pragma unroll
    for (int u = 0; u < kScanChunk / kScanSub; ++u) {
        start[u] = s;
        for (int i = 0; i < kScanSub; ++i) {
            const int64_t t = k.t0 + u * kScanSub + i;
            if (t >= k.end) break;
            const int64_t row = t * p.B + k.b;
            const float d = sigmoid_neg(at<V>(p.gate, row, p.ldg, k.c) + k.bias);
            s = s + fmaf(-d, s, input_factor<IN>(d) * at<V>(p.x, row, p.ldx, k.c));
        }
    }
    float c = p.chunks > 1 ? p.mul[j * R + k.r] : p.dfinal ? p.dfinal[k.r] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int u = kScanChunk / kScanSub - 1; u >= 0; --u) {
        float before[kScanSub], dv[kScanSub], xv[kScanSub];
        s = start[u];
#pragma unroll
        for (int i = 0; i < kScanSub; ++i) {
            const int64_t t = k.t0 + u * kScanSub + i;
            before[i] = s;
            dv[i] = xv[i] = 0.f;
            if (t < k.end) {
                const int64_t row = t * p.B + k.b;
                dv[i] = sigmoid_neg(at<V>(p.gate, row, p.ldg, k.c) + k.bias);
                xv[i] = at<V>(p.x, row, p.ldx, k.c);
                s = s + fmaf(-dv[i], s, input_factor<IN>(dv[i]) * xv[i]);
            }
        }
#pragma unroll
        for (int i = kScanSub - 1; i >= 0; --i) {
            const int64_t t = k.t0 + u * kScanSub + i;
            if (t < k.end) {
                const int64_t row = t * p.B + k.b;
                const float g = at<V>(p.dy, row, p.lddy, k.c) + c;
                const float dz = g * gate_slope<IN>(dv[i], xv[i], before[i]);
                dx[row * p.lddx + k.c] = (V)(g * input_factor<IN>(dv[i]));
                dg[row * p.lddg + k.c] = (V)dz;
                sum += dz;
                c = fmaf(-dv[i], g, g);
            }
        }
    }
    if (p.pbias) p.pbias[j * R + k.r] = sum;
    if (p.dstate && j == 0) p.dstate[k.r] = c;
}

// dbias: the chunks' and rows' partial sums of one channel, in a fixed order.
__global__ void __launch_bounds__(64) k_scan_dbias(ScanArgs p, float *dbias) {
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= p.D) return;
    float sum = 0.f;
    for (int64_t i = 0; i < (int64_t)p.chunks * p.B; ++i) sum += p.pbias[i * p.D + c];
    dbias[c] = sum;
}

// T = 0: the state passes through.
__global__ void __launch_bounds__(64) k_scan_pass(const float *from, float *to, size_t n) {
    const size_t i = blockIdx.x * (size_t)64 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.f;
}

struct Plan {
    size_t R;
    int64_t chunks;
    size_t part;       // bytes of one [chunks][R] array
};

const char *scan_plan(const fi_scan_desc *q, Plan &p) {
    if (!q) return "null descriptor";
    if (q->T < 0 || q->batch < 1 || q->channels < 1) return "T >= 0, batch >= 1 and channels >= 1 are needed";
    if (!value_type(q->dtype)) return "dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->input < FI_SCAN_PLAIN || q->input > FI_SCAN_ENERGY) return "input is none of FI_SCAN_*";
    const int64_t ld[] = {q->ld_x, q->ld_gate, q->ld_y, q->ld_dy, q->ld_dx, q->ld_dgate};
    for (int64_t v : ld)
        if (v != 0 && (v < q->channels || v > (int64_t(1) << 40))) return "a row pitch is less than channels";
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    p.R = (size_t)q->batch * q->channels;
    if (p.R > (size_t(1) << 24)) return "batch * channels is over 2^24";
    if (q->T > (int64_t(1) << 23)) return "T is over 2^23";
    p.chunks = (q->T + kScanChunk - 1) / kScanChunk;
    if (p.chunks > 65535) return "too many chunks";
    p.part = up256((size_t)p.chunks * p.R * sizeof(float));
    return nullptr;
}

size_t scan_workspace(const Plan &p, bool backward) {
    return std::max<size_t>(backward ? p.part * 3 : p.chunks > 1 ? p.part * 2 : 0, 256);
}

void scan_args(const fi_scan_desc *q, const Plan &pl, ScanArgs &a) {
    a.T = q->T;
    a.B = q->batch;
    a.D = q->channels;
    a.chunks = (int)pl.chunks;
    a.ldx = pitch_or(q->ld_x, a.D);
    a.ldg = pitch_or(q->ld_gate, a.D);
    a.ldy = pitch_or(q->ld_y, a.D);
    a.lddy = pitch_or(q->ld_dy, a.D);
    a.lddx = pitch_or(q->ld_dx, a.D);
    a.lddg = pitch_or(q->ld_dgate, a.D);
}

template <typename V, int IN>
void scan_forward(const ScanArgs &a, hipStream_t st) {
    const dim3 cols((unsigned)((a.B * (size_t)a.D + 63) / 64)), grid(cols.x, (unsigned)a.chunks);
    float *ends = a.saved;
    if (a.chunks > 1) {
        hipLaunchKernelGGL((k_scan_map<V, IN>), grid, dim3(64), 0, st, a);
        if (!ends) ends = a.add;
        hipLaunchKernelGGL(k_scan_carry, cols, dim3(64), 0, st, a, ends);
    }
    hipLaunchKernelGGL((k_scan_apply<V, IN>), grid, dim3(64), 0, st, a, (const float *)ends);
}

template <typename V, int IN>
void scan_backward(const ScanArgs &a, hipStream_t st) {
    const dim3 cols((unsigned)((a.B * (size_t)a.D + 63) / 64)), grid(cols.x, (unsigned)a.chunks);
    if (a.chunks > 1) {
        hipLaunchKernelGGL((k_scan_bmap<V>), grid, dim3(64), 0, st, a);
        hipLaunchKernelGGL(k_scan_bcarry, cols, dim3(64), 0, st, a);
    }
    hipLaunchKernelGGL((k_scan_bapply<V, IN>), grid, dim3(64), 0, st, a);
}

using ScanLaunch = void (*)(const ScanArgs &, hipStream_t);

template <typename V>
ScanLaunch pick(int input, bool backward) {
    switch (input) {
        case FI_SCAN_PLAIN: return backward ? &scan_backward<V, FI_SCAN_PLAIN> : &scan_forward<V, FI_SCAN_PLAIN>;
        case FI_SCAN_CONVEX: return backward ? &scan_backward<V, FI_SCAN_CONVEX> : &scan_forward<V, FI_SCAN_CONVEX>;
        default: return backward ? &scan_backward<V, FI_SCAN_ENERGY> : &scan_forward<V, FI_SCAN_ENERGY>;
    }
}

ScanLaunch pick(int dtype, int input, bool backward) {
    return dtype == FI_F32 ? pick<float>(input, backward)
                           : dtype == FI_BF16 ? pick<bf16_t>(input, backward) : pick<f16_t>(input, backward);
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_scan_saved_bytes(const fi_scan_desc *desc) {
    Plan pl;
    return scan_plan(desc, pl) ? 0 : std::max<size_t>(pl.part, 256);
}

size_t fi_scan_workspace_bytes(const fi_scan_desc *desc, int backward) {
    Plan pl;
    if (scan_plan(desc, pl)) return 0;
    return scan_workspace(pl, backward);
}

fi_status fi_scan_forward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                          const float *state, const int32_t *lengths, void *y, float *final, void *saved,
                          void *workspace, void *stream) {
    static const char *call = "fi_scan_forward";
    Plan pl;
    if (const char *why = scan_plan(desc, pl)) return op_fail(FI_EINVAL, call, why);
    const hipStream_t st = (hipStream_t)stream;
    ScanArgs a = {};
    scan_args(desc, pl, a);
    const size_t es = value_bytes(desc->dtype), w = a.D * es, fr = pl.R * sizeof(float);
    const int64_t rows = desc->T * a.B;
    const size_t ws = scan_workspace(pl, false);
    if (rows > 0 && (!x || !gate || !y || (!workspace && ws > 256)))
        return op_fail(FI_EINVAL, call, "x, gate, y and workspace are required");
    if ((uintptr_t)workspace % 256 || (uintptr_t)saved % 256)
        return op_fail(FI_EINVAL, call, "workspace and saved need an alignment of 256 bytes");
    const View out[] = {{y, rows, w, a.ldy * es}, {final, 1, fr, fr}, {saved, 1, pl.part, pl.part},
                        {workspace, 1, ws, ws}};
    const View in[] = {{x, rows, w, a.ldx * es}, {gate, rows, w, a.ldg * es}, {bias, 1, a.D * 4u, a.D * 4u},
                       {lengths, 1, a.B * 4u, a.B * 4u}, {final == state ? nullptr : state, 1, fr, fr}};
    if (outputs_meet(out, 4, in, 5) || (final == state && views_meet({state, 1, fr, fr}, out[0])))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    a.x = x, a.gate = gate, a.bias = bias, a.state = state, a.lengths = lengths;
    a.y = y, a.final = final, a.saved = (float *)saved;
    if (rows == 0) {
        if (final && final != state)
            hipLaunchKernelGGL(k_scan_pass, dim3((unsigned)((pl.R + 63) / 64)), dim3(64), 0, st, state, final, pl.R);
        return op_launched(call);
    }
    a.mul = (float *)workspace;
    a.add = (float *)((char *)workspace + pl.part);
    pick(desc->dtype, desc->input, false)(a, st);
    return op_launched(call);
}

fi_status fi_scan_backward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                           const float *state, const int32_t *lengths, const void *saved, const void *dy,
                           const float *dfinal, void *dx, void *dgate, float *dbias, float *dstate,
                           void *workspace, void *stream) {
    static const char *call = "fi_scan_backward";
    Plan pl;
    if (const char *why = scan_plan(desc, pl)) return op_fail(FI_EINVAL, call, why);
    const hipStream_t st = (hipStream_t)stream;
    ScanArgs a = {};
    scan_args(desc, pl, a);
    const size_t es = value_bytes(desc->dtype), w = a.D * es, fr = pl.R * sizeof(float);
    const int64_t rows = desc->T * a.B;
    if (rows > 0 && (!x || !gate || !saved || !dy || !dx || !dgate || !workspace))
        return op_fail(FI_EINVAL, call, "x, gate, saved, dy, dx, dgate and workspace are required");
    if ((uintptr_t)workspace % 256 || (uintptr_t)saved % 256)
        return op_fail(FI_EINVAL, call, "workspace and saved need an alignment of 256 bytes");
    const size_t ws = scan_workspace(pl, true);
    const View out[] = {{dx, rows, w, a.lddx * es}, {dgate, rows, w, a.lddg * es}, {dbias, 1, a.D * 4u, a.D * 4u},
                        {dstate, 1, fr, fr}, {workspace, 1, ws, ws}};
    const View in[] = {{x, rows, w, a.ldx * es}, {gate, rows, w, a.ldg * es}, {dy, rows, w, a.lddy * es},
                       {bias, 1, a.D * 4u, a.D * 4u}, {lengths, 1, a.B * 4u, a.B * 4u}, {state, 1, fr, fr},
                       {dfinal, 1, fr, fr}, {saved, 1, pl.part, pl.part}};
    if (outputs_meet(out, 5, in, 8)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    a.x = x, a.gate = gate, a.bias = bias, a.state = state, a.lengths = lengths;
    a.saved = (float *)saved, a.dy = dy, a.dfinal = dfinal, a.dx = dx, a.dgate = dgate, a.dstate = dstate;
    const unsigned cols = (unsigned)((pl.R + 63) / 64);
    if (rows == 0) {
        if (dstate) hipLaunchKernelGGL(k_scan_pass, dim3(cols), dim3(64), 0, st, dfinal, dstate, pl.R);
    } else {
        a.mul = (float *)workspace;
        a.add = (float *)((char *)workspace + pl.part);
        a.pbias = dbias ? (float *)((char *)workspace + 2 * pl.part) : nullptr;
        pick(desc->dtype, desc->input, true)(a, st);
    }
    if (dbias) hipLaunchKernelGGL(k_scan_dbias, dim3((unsigned)((a.D + 63) / 64)), dim3(64), 0, st, a, dbias);
    return op_launched(call);
}

}  // extern "C"
