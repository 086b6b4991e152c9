// The norms around a block, fused with its gate, residual and residual scale
// (fi_norm_*).  Per row of D values:
//   v = o q w1, q = 1/sqrt(mean o^2 + eps);  m = v act(g);  r = res + k m;
//   a = r p w2, p = 1/sqrt(mean r^2 + eps).
// Backwards, with u = da w2:
//   dR = dr + p (u - r p mean(u r p)),  dm = k dR,  dv = dm act(g),
//   dg = dm v act'(g),  do = q (dv w1 - o q mean(dv w1 o q)),
//   dk = sum m dR, dw1 = sum dv o q, dw2 = sum da r p   (over the rows).
// r is formed again from o, g and res in fp32, not read back rounded.
#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 16384;
constexpr int kNormGroups = 1024;      // workgroups of the backward pass at most, each with its own column sums

struct NormArgs {
    const void *o, *gate, *res, *dr, *da;
    void *r, *a, *d_o, *dgate, *dres;
    const float *w1, *k, *w2;
    float *saved;            // [2][rows]
    float *part;             // [groups][3][D] column sums of dw1, dk, dw2
    int64_t rows;
    int64_t ldo, ldg, ldres, ldr, lda, lddr, ldda, lddo, lddg, lddres;
    int D;
    int post, act;
    float eps;
    bool col1, colk, col2;   // column sums wanted
};

__device__ __forceinline__ float block_sum(float v, float *lds) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += lds[i];
    return s;
}

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896f));
}

// act(g) and its derivative
__device__ __forceinline__ float act_of(int act, float g, float &slope) {
    if (act == FI_GATE_LINEAR) {
        slope = 1.f;
        return g;
    }
    const float s = sigmoid(g);
    if (act == FI_GATE_SIGMOID) {
        slope = s * (1.f - s);
        return s;
    }
    slope = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
}

template <typename V>
__device__ __forceinline__ float ld(const void *p, int64_t i) {
    return (float)static_cast<const V *>(p)[i];
}

// One element's m (and what the backward pass needs of it).
template <typename V>
__device__ __forceinline__ float block_out(const NormArgs &p, int64_t row, int c, float q, float &unit, float &act,
                                           float &slope) {
    unit = act = slope = 0.f;
    if (!p.o) return 0.f;
    unit = ld<V>(p.o, row * p.ldo + c) * q;
    float v = unit * (p.w1 ? p.w1[c] : 1.f);
    act = 1.f;
    if (p.gate) act = act_of(p.act, ld<V>(p.gate, row * p.ldg + c), slope);
    return v * act;
}

template <typename V, typename W>
__device__ __forceinline__ float stream_out(const NormArgs &p, int64_t row, int c, float m) {
    const float r = p.res ? ld<W>(p.res, row * p.ldres + c) : 0.f;
    return p.o ? fmaf(p.k ? p.k[c] : 1.f, m, r) : r;
}

template <typename V, typename W>
__global__ void __launch_bounds__(kNormThreads) k_norm(NormArgs p) {
    __shared__ float lds[kNormThreads / 64];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float q = 1.f, unit, act, slope;
        if (p.post) {
            float s = 0.f;
            for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
                const float v = ld<V>(p.o, row * p.ldo + c);
                s = fmaf(v, v, s);
            }
            q = 1.f / sqrtf(block_sum(s, lds) / (float)p.D + p.eps);
        }
        float s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
            const float r = stream_out<V, W>(p, row, c, block_out<V>(p, row, c, q, unit, act, slope));
            s = fmaf(r, r, s);
        }
        const float n = 1.f / sqrtf(block_sum(s, lds) / (float)p.D + p.eps);
        for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
            const float r = stream_out<V, W>(p, row, c, block_out<V>(p, row, c, q, unit, act, slope));
            if (p.r) static_cast<W *>(p.r)[row * p.ldr + c] = (W)r;
            if (p.a) static_cast<V *>(p.a)[row * p.lda + c] = (V)(r * n * (p.w2 ? p.w2[c] : 1.f));
        }
        if (p.saved && threadIdx.x == 0) {
            p.saved[row] = q;
            p.saved[p.rows + row] = n;
        }
    }
}

template <typename V, typename W>
__global__ void __launch_bounds__(kNormThreads) k_norm_back(NormArgs p) {
    __shared__ float lds[kNormThreads / 64];
    float *part = p.part + (size_t)blockIdx.x * 3 * p.D;
    for (int c = threadIdx.x; c < 3 * p.D; c += kNormThreads) part[c] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float q = p.post ? p.saved[row] : 1.f, n = p.saved[p.rows + row];
        float unit, act, slope;
        float mean2 = 0.f;
        if (p.da) {
            float s = 0.f;
            for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
                const float r = stream_out<V, W>(p, row, c, block_out<V>(p, row, c, q, unit, act, slope));
                s = fmaf(ld<V>(p.da, row * p.ldda + c) * (p.w2 ? p.w2[c] : 1.f), r * n, s);
            }
            mean2 = block_sum(s, lds) / (float)p.D;
        }
        // dR at one element, and its unit r
        const auto grad = [&](int c, float m, float &da, float &ru) {
            const float r = stream_out<V, W>(p, row, c, m);
            float g = p.dr ? ld<W>(p.dr, row * p.lddr + c) : 0.f;
            da = 0.f;
            ru = r * n;
            if (p.da) {
                da = ld<V>(p.da, row * p.ldda + c);
                g = fmaf(n, fmaf(-ru, mean2, da * (p.w2 ? p.w2[c] : 1.f)), g);
            }
            return g;
        };
        float mean1 = 0.f;
        if (p.post && p.d_o) {
            float s = 0.f;
            for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
                float da, ru;
                const float m = block_out<V>(p, row, c, q, unit, act, slope);
                const float dm = grad(c, m, da, ru) * (p.k ? p.k[c] : 1.f);
                s = fmaf(dm * act * (p.w1 ? p.w1[c] : 1.f), unit, s);
            }
            mean1 = block_sum(s, lds) / (float)p.D;
        }
        __syncthreads();   // dres may be dr: every read of the row is done
        for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
            float da, ru;
            const float m = block_out<V>(p, row, c, q, unit, act, slope);
            const float g = grad(c, m, da, ru);
            const float w1 = p.w1 ? p.w1[c] : 1.f;
            const float dm = g * (p.k ? p.k[c] : 1.f);
            const float dv = dm * act;
            if (p.dres) static_cast<W *>(p.dres)[row * p.lddres + c] = (W)g;
            if (p.dgate) static_cast<V *>(p.dgate)[row * p.lddg + c] = (V)(dm * unit * w1 * slope);
            if (p.d_o)
                static_cast<V *>(p.d_o)[row * p.lddo + c] = (V)(p.post ? q * fmaf(-unit, mean1, dv * w1) : dv * w1);
            if (p.col1) part[c] = fmaf(dv, unit, part[c]);
            if (p.colk) part[p.D + c] = fmaf(m, g, part[p.D + c]);
            if (p.col2) part[2 * p.D + c] = fmaf(da, ru, part[2 * p.D + c]);
        }
    }
}

// The workgroups' column sums, in their order.
__global__ void __launch_bounds__(64) k_norm_columns(const float *part, int groups, int D, float *dw1, float *dk,
                                                     float *dw2) {
    const int i = blockIdx.x * 64 + threadIdx.x;
    if (i >= 3 * D) return;
    float *to = i < D ? dw1 : i < 2 * D ? dk : dw2;
    if (!to) return;
    float s = 0.f;
    for (int g = 0; g < groups; ++g) s += part[(size_t)g * 3 * D + i];
    to[i % D] = s;
}

const char *norm_check(const fi_norm_desc *q) {
    if (!q) return "null descriptor";
    if (q->rows < 0 || q->rows > (int64_t(1) << 40)) return "rows is negative or over 2^40";
    if (q->channels < 1 || q->channels > kNormMaxD) return "channels is not in 1 .. 16384";
    if (!value_type(q->dtype)) return "dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->res_dtype != q->dtype && q->res_dtype != FI_F32) return "res_dtype is neither dtype nor FI_F32";
    if (q->post_norm != 0 && q->post_norm != 1) return "post_norm is not 0 or 1";
    if (q->act < FI_GATE_LINEAR || q->act > FI_GATE_SILU) return "act is none of FI_GATE_*";
    if (!(q->eps >= 0.f)) return "eps is negative or not a number";
    const int64_t ld[] = {q->ld_o, q->ld_gate, q->ld_res, q->ld_r, q->ld_a,
                          q->ld_dr, q->ld_da, q->ld_do, q->ld_dgate, q->ld_dres};
    for (int64_t v : ld)
        if (v != 0 && (v < q->channels || v > (int64_t(1) << 40))) return "a row pitch is less than channels";
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    return nullptr;
}

int norm_groups(int64_t rows) { return (int)(rows < kNormGroups ? (rows < 1 ? 1 : rows) : kNormGroups); }

int64_t pitch(int64_t ld, int64_t width) { return ld ? ld : width; }

void norm_args(const fi_norm_desc *q, NormArgs &a) {
    a.rows = q->rows;
    a.D = q->channels;
    a.post = q->post_norm;
    a.act = q->act;
    a.eps = q->eps;
    a.ldo = pitch(q->ld_o, a.D);
    a.ldg = pitch(q->ld_gate, a.D);
    a.ldres = pitch(q->ld_res, a.D);
    a.ldr = pitch(q->ld_r, a.D);
    a.lda = pitch(q->ld_a, a.D);
    a.lddr = pitch(q->ld_dr, a.D);
    a.ldda = pitch(q->ld_da, a.D);
    a.lddo = pitch(q->ld_do, a.D);
    a.lddg = pitch(q->ld_dgate, a.D);
    a.lddres = pitch(q->ld_dres, a.D);
}

template <typename V, typename W>
void launch(const NormArgs &a, bool backward, unsigned groups, hipStream_t st) {
    if (backward)
        hipLaunchKernelGGL((k_norm_back<V, W>), dim3(groups), dim3(kNormThreads), 0, st, a);
    else
        hipLaunchKernelGGL((k_norm<V, W>), dim3(groups), dim3(kNormThreads), 0, st, a);
}

void launch(const fi_norm_desc *q, const NormArgs &a, bool backward, unsigned groups, hipStream_t st) {
    if (q->dtype == FI_F32) launch<float, float>(a, backward, groups, st);
    else if (q->dtype == FI_BF16)
        q->res_dtype == FI_F32 ? launch<bf16_t, float>(a, backward, groups, st)
                               : launch<bf16_t, bf16_t>(a, backward, groups, st);
    else
        q->res_dtype == FI_F32 ? launch<f16_t, float>(a, backward, groups, st)
                               : launch<f16_t, f16_t>(a, backward, groups, st);
}

// The inputs that both passes take; an error message or nullptr.
const char *norm_inputs(const fi_norm_desc *q, const void *o, const void *gate, const void *res, const float *w1,
                        const float *k) {
    if (q->rows == 0) return nullptr;
    if (!o && !res) return "o or res is required";
    if (!o && (gate || w1 || k || q->post_norm)) return "gate, post_weight, scale and post_norm need o";
    if (w1 && !q->post_norm) return "post_weight needs post_norm";
    return nullptr;
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_norm_workspace_bytes(const fi_norm_desc *desc) {
    if (norm_check(desc)) return 0;
    return up256((size_t)norm_groups(desc->rows) * 3 * desc->channels * sizeof(float));
}

fi_status fi_norm_forward(const fi_norm_desc *desc, const void *o, const void *gate, const void *res,
                          const float *post_weight, const float *scale, const float *pre_weight, void *r, void *a,
                          float *saved, void *stream) {
    static const char *call = "fi_norm_forward";
    if (const char *why = norm_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (const char *why = norm_inputs(desc, o, gate, res, post_weight, scale)) return op_fail(FI_EINVAL, call, why);
    if (desc->rows == 0 || (!r && !a && !saved)) return FI_OK;
    NormArgs n = {};
    norm_args(desc, n);
    const size_t es = value_bytes(desc->dtype), rs = value_bytes(desc->res_dtype), D = n.D;
    const View vr = {r, n.rows, D * rs, n.ldr * rs}, vres = {res, n.rows, D * rs, n.ldres * rs};
    const View out[] = {vr, {a, n.rows, D * es, n.lda * es}, {saved, 1, (size_t)n.rows * 8, (size_t)n.rows * 8}};
    const View in[] = {{o, n.rows, D * es, n.ldo * es}, {gate, n.rows, D * es, n.ldg * es},
                       {post_weight, 1, D * 4, D * 4}, {scale, 1, D * 4, D * 4}, {pre_weight, 1, D * 4, D * 4}};
    const bool inplace = same_view(vr, vres);
    if (outputs_meet(out, 3, in, 5) || outputs_meet(out + 1, 2, &vres, 1) || (!inplace && views_meet(vr, vres)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    n.o = o, n.gate = gate, n.res = res, n.w1 = post_weight, n.k = scale, n.w2 = pre_weight;
    n.r = r, n.a = a, n.saved = saved;
    launch(desc, n, false, (unsigned)std::min<int64_t>(n.rows, 1 << 20), (hipStream_t)stream);
    return op_launched(call);
}

fi_status fi_norm_backward(const fi_norm_desc *desc, const void *o, const void *gate, const void *res,
                           const float *post_weight, const float *scale, const float *pre_weight, const float *saved,
                           const void *dr, const void *da, void *d_o, void *dgate, void *dres, float *dpost,
                           float *dscale, float *dpre, void *workspace, void *stream) {
    static const char *call = "fi_norm_backward";
    if (const char *why = norm_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (const char *why = norm_inputs(desc, o, gate, res, post_weight, scale)) return op_fail(FI_EINVAL, call, why);
    NormArgs n = {};
    norm_args(desc, n);
    if (n.rows > 0) {
        if (!saved || !workspace || (uintptr_t)workspace % 256)
            return op_fail(FI_EINVAL, call, "saved and a workspace aligned to 256 bytes are required");
        if ((d_o && !o) || (dgate && !gate) || (dres && !res) || (dpost && !n.post) || (dscale && !o) || (dpre && !da))
            return op_fail(FI_EINVAL, call, "a gradient is asked for whose input is not given");
    }
    const size_t es = value_bytes(desc->dtype), rs = value_bytes(desc->res_dtype), D = n.D;
    const size_t ws = fi_norm_workspace_bytes(desc);
    const View vdr = {dr, n.rows, D * rs, n.lddr * rs}, vdres = {dres, n.rows, D * rs, n.lddres * rs};
    const View out[] = {vdres, {d_o, n.rows, D * es, n.lddo * es}, {dgate, n.rows, D * es, n.lddg * es},
                        {dpost, 1, D * 4, D * 4}, {dscale, 1, D * 4, D * 4}, {dpre, 1, D * 4, D * 4},
                        {workspace, 1, ws, ws}};
    const View in[] = {{o, n.rows, D * es, n.ldo * es}, {gate, n.rows, D * es, n.ldg * es},
                       {res, n.rows, D * rs, n.ldres * rs}, {da, n.rows, D * es, n.ldda * es},
                       {post_weight, 1, D * 4, D * 4}, {scale, 1, D * 4, D * 4}, {pre_weight, 1, D * 4, D * 4},
                       {saved, 1, (size_t)n.rows * 8, (size_t)n.rows * 8}};
    const bool inplace = same_view(vdr, vdres);
    if (outputs_meet(out, 7, in, 8) || outputs_meet(out + 1, 6, &vdr, 1) || (!inplace && views_meet(vdr, vdres)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    n.o = o, n.gate = gate, n.res = res, n.w1 = post_weight, n.k = scale, n.w2 = pre_weight;
    n.saved = (float *)saved, n.dr = dr, n.da = da, n.d_o = d_o, n.dgate = dgate, n.dres = dres;
    n.part = (float *)workspace, n.col1 = dpost, n.colk = dscale, n.col2 = dpre;
    const hipStream_t st = (hipStream_t)stream;
    const int groups = n.rows > 0 ? norm_groups(n.rows) : 0;
    if (groups) launch(desc, n, true, (unsigned)groups, st);
    if (dpost || dscale || dpre)
        hipLaunchKernelGGL(k_norm_columns, dim3((unsigned)((3 * D + 63) / 64)), dim3(64), 0, st, (const float *)workspace,
                           groups, n.D, dpost, dscale, dpre);
    return op_launched(call);
}

}  // extern "C"
