// The norms around a block, fused with its gate, residual and residual scale
// (fi_norm_*).  Per row of D values:
//   v = o q w1, q = 1/sqrt(mean o^2 + eps);  m = v act(g);  r = res + k m;
//   a = r p w2, p = 1/sqrt(mean r^2 + eps).
// Backwards, with u = da w2:
//   dR = dr + p (u - r p mean(u r p)),  dm = k dR,  dv = dm act(g),
//   dg = dm v act'(g),  do = q (dv w1 - o q mean(dv w1 o q)),
//   dw1 = k P, dk = w1 P with P = sum dR act(g) o q,  dw2 = sum da r p   (over the rows).
// r is formed again from o, g and res in fp32, not read back rounded.
#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormLane = 16;          // values of a row per lane at most
constexpr int kNormForwardGroups = 2048;
constexpr int kNormGroups = 512;       // workgroups of the backward pass at most, each with its own column sums

struct NormArgs {
    const void *o, *gate, *res, *dr, *da;
    void *r, *a, *d_o, *dgate, *dres;
    const float *w1, *k, *w2;
    float *saved;            // [2][rows]
    float *part;             // [groups][2][D] column sums of dR act o q and of da r p
    int64_t rows;
    int64_t ldo, ldg, ldres, ldr, lda, lddr, ldda, lddo, lddg, lddres;
    int D;
    int post, act;
    float eps;
    bool columns;            // column sums wanted
};

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

// A row is held in registers by a team: one wave up to 1024 values (four teams
// to a workgroup, no barrier), else a workgroup of as many waves as the row
// needs.  A lane holds NC chunks of CH neighbouring values, CH chosen so that
// the widest tensor of the row is read 16 bytes at a time; a team's waves take
// alternate stretches.  A team keeps its columns' weights (and, backwards,
// their column sums) in registers over all its rows.
template <int CH, int NC, bool MULTI>
struct Team {
    int start, step;       // first column of this lane, columns between its chunks
    int waves, wave, lane;
    int64_t row, rows_step;
    int turn;

    __device__ __forceinline__ Team() {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = blockDim.x >> 6;
        turn = 0;
        if (MULTI) {
            start = (wave * 64 + lane) * CH;
            step = waves * 64 * CH;
            row = blockIdx.x;
            rows_step = gridDim.x;
        } else {
            start = lane * CH;
            step = 64 * CH;
            row = blockIdx.x * (int64_t)waves + wave;
            rows_step = gridDim.x * (int64_t)waves;
        }
    }
    // Sum over the team, in every lane.  Two sets of slots by turns: a wave that
    // writes a set has passed the barrier after everybody's reads of that set.
    __device__ __forceinline__ float sum(float v, float (*slots)[16]) {
        v = lanes_sum(v);
        if (!MULTI) return v;
        if (lane == 0) slots[turn][wave] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < waves; ++i) v += slots[turn][i];
        turn ^= 1;
        return v;
    }
};

template <typename T, int CH, int NC, bool MULTI>
__device__ __forceinline__ void load_row(float (&v)[NC * CH], const void *p, int64_t ld, const Team<CH, NC, MULTI> &t,
                                         int D) {
    const T *from = static_cast<const T *>(p) + t.row * ld;
    Chunk<T, CH> raw[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = t.start + j * t.step;
        raw[j] = load_chunk<T, CH>(from + c, D - c);
    }
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j * CH + i] = (float)raw[j][i];
}

template <typename T, int CH, int NC, bool MULTI>
__device__ __forceinline__ void store_row(const float (&v)[NC * CH], void *p, int64_t ld,
                                          const Team<CH, NC, MULTI> &t, int D) {
    T *to = static_cast<T *>(p) + t.row * ld;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = t.start + j * t.step;
        Chunk<T, CH> raw;
#pragma unroll
        for (int i = 0; i < CH; ++i) raw[i] = (T)v[j * CH + i];
        store_chunk<T, CH>(to + c, D - c, raw);
    }
}

template <int CH, int NC, bool MULTI>
__device__ __forceinline__ void load_weights(float (&v)[NC * CH], const float *w, const Team<CH, NC, MULTI> &t,
                                             int D) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = t.start + j * t.step;
        Chunk<float, CH> raw;
        if (w) raw = load_chunk<float, CH>(w + c, D - c);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j * CH + i] = w ? raw[i] : 1.f;
    }
}

// k w1: the two weights of a column meet in every use of them in a row
template <int CH, int NC, bool MULTI>
__device__ __forceinline__ void load_product(float (&v)[NC * CH], const float *k, const float *w1,
                                             const Team<CH, NC, MULTI> &t, int D) {
    float w[NC * CH];
    load_weights(v, k, t, D);
    load_weights(w, w1, t, D);
#pragma unroll
    for (int i = 0; i < NC * CH; ++i) v[i] *= w[i];
}

__device__ __forceinline__ float rnorm(float squares, const NormArgs &p) {
    return 1.f / sqrtf(squares / (float)p.D + p.eps);
}

// Forward: HBM-bound, every tensor once.
template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm(NormArgs p) {
    constexpr int N = CH * NC;
    __shared__ float slots[2][16];
    Team<CH, NC, MULTI> t;
    float kw[N], w2[N];
    load_product(kw, p.k, p.w1, t, p.D);
    load_weights(w2, p.w2, t, p.D);
    for (; t.row < p.rows; t.row += t.rows_step) {
        float o[N], g[N], r[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = 0.f, g[i] = 0.f, r[i] = 0.f;
        if (p.o) load_row<V>(o, p.o, p.ldo, t, p.D);
        if (p.gate) load_row<V>(g, p.gate, p.ldg, t, p.D);
        if (p.res) load_row<W>(r, p.res, p.ldres, t, p.D);
        float q = 1.f;
        if (p.post) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(o[i], o[i], s);
            q = rnorm(t.sum(s, slots), p);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float m = o[i] * q;
            if (p.gate) {
                float slope;
                m *= act_of(p.act, g[i], slope);
            }
            r[i] = fmaf(kw[i], m, r[i]);
            s = fmaf(r[i], r[i], s);
        }
        const float n = rnorm(t.sum(s, slots), p);
        if (p.r) store_row<W>(r, p.r, p.ldr, t, p.D);
        if (p.a) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = r[i] * n * w2[i];
            store_row<V>(r, p.a, p.lda, t, p.D);
        }
        if (p.saved && (t.start == 0)) {
            p.saved[t.row] = q;
            p.saved[p.rows + t.row] = n;
        }
    }
}

// Backward: every tensor of the row once, two row means, one after the other;
// the column sums of a team's rows in registers, its workgroup's joined in LDS
// (team after team, so the order is fixed) and written once.
template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm_back(NormArgs p) {
    constexpr int N = CH * NC;
    __shared__ float slots[2][16];
    __shared__ float join[MULTI ? 1 : 2 * 64 * N];
    Team<CH, NC, MULTI> t;
    float kw[N], w2[N], c1[N], c2[N];
    load_product(kw, p.k, p.w1, t, p.D);
    load_weights(w2, p.w2, t, p.D);
#pragma unroll
    for (int i = 0; i < N; ++i) c1[i] = c2[i] = 0.f;
    for (; t.row < p.rows; t.row += t.rows_step) {
        float o[N], g[N], r[N], dr[N], da[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = g[i] = r[i] = dr[i] = da[i] = 0.f;
        if (p.o) load_row<V>(o, p.o, p.ldo, t, p.D);
        if (p.gate) load_row<V>(g, p.gate, p.ldg, t, p.D);
        if (p.res) load_row<W>(r, p.res, p.ldres, t, p.D);
        if (p.da) load_row<V>(da, p.da, p.ldda, t, p.D);
        if (p.dr) load_row<W>(dr, p.dr, p.lddr, t, p.D);
        const float q = p.post ? p.saved[t.row] : 1.f, n = p.saved[p.rows + t.row];
        float act[N];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            o[i] *= q;                                   // unit o
            float slope = 0.f;
            act[i] = 1.f;
            if (p.gate) act[i] = act_of(p.act, g[i], slope);
            g[i] = slope;
            r[i] = fmaf(kw[i], o[i] * act[i], r[i]) * n;   // unit r
            c2[i] = fmaf(da[i], r[i], c2[i]);
            da[i] *= w2[i];
            s = fmaf(da[i], r[i], s);
        }
        const float mean2 = p.da ? t.sum(s, slots) / (float)p.D : 0.f;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dr[i] = fmaf(n, fmaf(-r[i], mean2, da[i]), dr[i]);   // dR
            const float e = dr[i] * act[i];
            c1[i] = fmaf(e, o[i], c1[i]);
            act[i] = e * kw[i];
            s = fmaf(act[i], o[i], s);
        }
        if (p.dres) store_row<W>(dr, p.dres, p.lddres, t, p.D);
        const float mean1 = p.post && p.d_o ? t.sum(s, slots) / (float)p.D : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] *= dr[i] * kw[i] * o[i];
            o[i] = p.post ? q * fmaf(-o[i], mean1, act[i]) : act[i];
        }
        if (p.dgate) store_row<V>(g, p.dgate, p.lddg, t, p.D);
        if (p.d_o) store_row<V>(o, p.d_o, p.lddo, t, p.D);
    }
    if (!p.columns) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
    if (!MULTI) {
        for (int w = 0; w < t.waves; ++w) {
            if (t.wave == w) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = i * 64 + t.lane;
                    if (w) c1[i] += join[at], c2[i] += join[64 * N + at];
                    join[at] = c1[i], join[64 * N + at] = c2[i];
                }
            }
            __syncthreads();
        }
        if (t.wave != t.waves - 1) return;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = t.start + j * t.step;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (c + i < p.D) {
                part[c + i] = c1[j * CH + i];
                part[p.D + c + i] = c2[j * CH + i];
            }
    }
}

// The workgroups' column sums: 64 columns a workgroup, its four waves take
// every fourth group and are added in their order.  dw1 and dk are the one sum
// of dR act o q times k and w1.
__global__ void __launch_bounds__(256) k_norm_columns(NormArgs p, int groups, float *dw1, float *dk, float *dw2) {
    __shared__ float join[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (i < 2 * p.D)
        for (int g = wave; g < groups; g += 4) s += p.part[(size_t)g * 2 * p.D + i];
    join[wave][lane] = s;
    __syncthreads();
    if (wave || i >= 2 * p.D) return;
    s = (join[0][lane] + join[1][lane]) + (join[2][lane] + join[3][lane]);
    if (i >= p.D) {
        if (dw2) dw2[i - p.D] = s;
        return;
    }
    if (dw1) dw1[i] = p.k ? p.k[i] * s : s;
    if (dk) dk[i] = p.w1 ? p.w1[i] * s : s;
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

// Waves of a team, and workgroups over `rows`: at most `most`, the rows spread evenly.
int team_waves(int D) { return (D + 64 * kNormLane - 1) / (64 * kNormLane); }

unsigned norm_groups(int64_t rows, int D, int64_t most) {
    const int64_t need = team_waves(D) > 1 ? rows : (rows + 3) / 4;
    if (need <= most) return (unsigned)(need < 1 ? 1 : need);
    const int64_t turns = (need + most - 1) / most;
    return (unsigned)((need + turns - 1) / turns);
}

void norm_args(const fi_norm_desc *q, NormArgs &a) {
    a.rows = q->rows;
    a.D = q->channels;
    a.post = q->post_norm;
    a.act = q->act;
    a.eps = q->eps;
    a.ldo = pitch_or(q->ld_o, a.D);
    a.ldg = pitch_or(q->ld_gate, a.D);
    a.ldres = pitch_or(q->ld_res, a.D);
    a.ldr = pitch_or(q->ld_r, a.D);
    a.lda = pitch_or(q->ld_a, a.D);
    a.lddr = pitch_or(q->ld_dr, a.D);
    a.ldda = pitch_or(q->ld_da, a.D);
    a.lddo = pitch_or(q->ld_do, a.D);
    a.lddg = pitch_or(q->ld_dgate, a.D);
    a.lddres = pitch_or(q->ld_dres, a.D);
}

template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS>
void launch(const NormArgs &a, bool backward, unsigned groups, unsigned threads, hipStream_t st) {
    if (backward)
        hipLaunchKernelGGL((k_norm_back<V, W, CH, NC, MULTI, THREADS>), dim3(groups), dim3(threads), 0, st, a);
    else
        hipLaunchKernelGGL((k_norm<V, W, CH, NC, MULTI, THREADS>), dim3(groups), dim3(threads), 0, st, a);
}

template <typename V, typename W>
void launch(const NormArgs &a, bool backward, unsigned groups, hipStream_t st) {
    constexpr int CH = sizeof(W) == 2 ? 8 : 4;
    const int waves = team_waves(a.D);
    if (a.D <= 64 * CH)
        launch<V, W, CH, 1, false, 256>(a, backward, groups, 256, st);
    else if (a.D <= 128 * CH)
        launch<V, W, CH, 2, false, 256>(a, backward, groups, 256, st);
    else if (waves == 1)
        launch<V, W, CH, kNormLane / CH, false, 256>(a, backward, groups, 256, st);
    else if (waves <= 8)
        launch<V, W, CH, kNormLane / CH, true, 512>(a, backward, groups, waves * 64, st);
    else
        launch<V, W, CH, kNormLane / CH, true, 1024>(a, backward, groups, waves * 64, st);
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
    return up256((size_t)norm_groups(desc->rows, desc->channels, kNormGroups) * 2 * desc->channels * sizeof(float));
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
    launch(desc, n, false, norm_groups(n.rows, n.D, kNormForwardGroups), (hipStream_t)stream);
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
    n.part = (float *)workspace, n.columns = dpost || dscale || dpre;
    const hipStream_t st = (hipStream_t)stream;
    const unsigned groups = n.rows > 0 ? norm_groups(n.rows, n.D, kNormGroups) : 0;
    if (groups) launch(desc, n, true, groups, st);
    if (n.columns)
        hipLaunchKernelGGL(k_norm_columns, dim3((unsigned)((2 * D + 63) / 64)), dim3(256), 0, st, n, (int)groups, dpost, dscale, dpre);
    return op_launched(call);
}

}  // extern "C"
