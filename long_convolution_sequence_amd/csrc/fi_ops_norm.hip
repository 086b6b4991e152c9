// The norms around a block, fused with its gate, residual and residual scale
// (fi_norm_*).  Per row of D values:
//   v = o q w1, q = 1/sqrt(mean o^2 + eps);  m = v act(g);  r = res + k m;
//   a = r p w2, p = 1/sqrt(mean r^2 + eps).
// Backwards, with u = da w2:
//   dR = dr + p (u - r p mean(u r p)),  dm = k dR,  dv = dm act(g),
//   dg = dm v act'(g),  do = q (dv w1 - o q mean(dv w1 o q)),
//   dw1 = k P, dk = w1 P with P = sum dR act(g) o q,  dw2 = sum da r p   (over the rows).
// r is formed again from o, g and res in fp32, not read back rounded.
#include "fi_rows.h"

namespace fi {

namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormHalf = 768;         // threads of the backward workgroups with half of that (see half_lanes)
constexpr int64_t kNormCache = 256 << 20;   // bytes of the last-level cache
constexpr int kNormCUs = 256;          // compute units that the workgroups are spread over

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

// act(g) and its derivative
__device__ __forceinline__ float act_of(int act, float g, float &slope) {
    if (act == FI_GATE_LINEAR) {
        slope = 1.f;
        return g;
    }
    const float t = __builtin_amdgcn_exp2f(g * -1.44269504088896f);     // e^-g
    const float s = __builtin_amdgcn_rcpf(1.f + t);
    if (act == FI_GATE_SIGMOID) {
        // 1 - s would lose the digits of what is left of an open gate's slope
        slope = s * (g > 0.f ? t * s : 1.f - s);
        return s;
    }
    slope = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
}

// A lane's weights: kw = k w1 (the two meet in every use of them in a row) and
// w2, 1 where none is given.  The loads do not wait for one another: a weight
// that is not given is read from another's place.  OWNED: 0 for an element that
// the lane does not own.
template <bool OWNED, int CH, int NC, bool MULTI>
__device__ __forceinline__ void load_weights(float (&kw)[NC * CH], float (&w2)[NC * CH], const NormArgs &p,
                                             const Team<CH, NC, MULTI> &t) {
    const float *any = p.w1 ? p.w1 : p.k ? p.k : p.w2;
    Chunk<float, CH> a[NC], b[NC], c[NC];
    if (any) {
        const float *pa = p.w1 ? p.w1 : any, *pb = p.k ? p.k : any, *pc = p.w2 ? p.w2 : any;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            a[j] = load_chunk<float, CH>(pa, t.at[j]);
            b[j] = load_chunk<float, CH>(pb, t.at[j]);
            c[j] = load_chunk<float, CH>(pc, t.at[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const bool own = !OWNED || i >= t.at[j].skip;
            kw[j * CH + i] = own ? (p.w1 ? a[j][i] : 1.f) * (p.k ? b[j][i] : 1.f) : 0.f;
            w2[j * CH + i] = own ? (p.w2 ? c[j][i] : 1.f) : 0.f;
        }
}

__device__ __forceinline__ float rnorm(float squares, const NormArgs &p) {
    return 1.f / sqrtf(squares / (float)p.D + p.eps);
}

// Forward: HBM-bound, every tensor once (131072 x 864 bf16 with fp32 rows 292 us, 5.4
// TB/s; 1999 x 5001 fp16 29 us, 2.8: few rows, a barrier in each).  A team of several waves reads its next
// row before it works on this one: a barrier a row holds all its waves, and few
// such teams fit a CU.  ALL: o, gate and res are there.  STREAM: the inputs are
// larger than the last-level cache (see launch).
template <typename V, typename W, int CH, int NC, bool MULTI, bool TAIL, bool ALL, bool STREAM, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm(NormArgs p) {
    constexpr int N = CH * NC;
    constexpr bool AHEAD = MULTI && THREADS <= 512;
    __shared__ float slots[2][16];
    Team<CH, NC, MULTI> t(p.D);
    Raw<ALL, STREAM, V, CH, NC> raw_o, raw_g;
    Raw<ALL, STREAM, W, CH, NC> raw_r;
    const auto fetch = [&](int64_t row) {
        raw_o.load(p.o, p.ldo, row, t);
        raw_g.load(p.gate, p.ldg, row, t);
        raw_r.load(p.res, p.ldres, row, t);
    };
    if (AHEAD && t.row < p.rows) fetch(t.row);
    float kw[N], w2[N];
    load_weights<false>(kw, w2, p, t);
    for (; t.row < p.rows; t.row += t.rows_step) {
        float o[N], g[N], r[N];
        if (!AHEAD) fetch(t.row);
        raw_o.get(o);
        raw_g.get(g);
        raw_r.get(r);
        if (AHEAD && t.row + t.rows_step < p.rows) fetch(t.row + t.rows_step);
        const float q = p.post ? rnorm(t.sum(squares<TAIL>(o, t), slots), p) : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float m = o[i] * q;
            if (ALL || p.gate) {
                float slope;
                m *= act_of(p.act, g[i], slope);
            }
            r[i] = fmaf(kw[i], m, r[i]);
        }
        const float n = rnorm(t.sum(squares<TAIL>(r, t), slots), p);
        if (p.r) store_row<TAIL, W>(r, p.r, p.ldr, t);
        if (p.a) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = r[i] * n * w2[i];
            store_row<TAIL, V>(r, p.a, p.lda, t);
        }
        if (p.saved && t.first) {
            p.saved[t.row] = q;
            p.saved[p.rows + t.row] = n;
        }
    }
}

// Backward: every tensor of the row once (131072 x 768 bf16 with fp32 rows 400 us, 5.5
// TB/s; 1999 x 5001 fp16 38 us), two row means, one after the other;
// the column sums of a team's rows in registers, its workgroup's joined in LDS
// (team after team, so the order is fixed) and written once.  Elements that a
// lane does not own have weights of zero, so both means pass them by.  Rows of more
// than 8192 values: 16 waves leave a lane 128 registers, 105 to 124 values of it
// spill, and that bounds it (2048 x 16384 bf16 with fp32 rows 409 us, 148 by its
// bytes; 2048 x 12288 338 and 111).
template <typename V, typename W, int CH, int NC, bool MULTI, bool TAIL, bool ALL, bool STREAM, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kNormHalf ? 3 : THREADS <= 512 ? 2 : 1) k_norm_back(NormArgs p) {
    constexpr int N = CH * NC;
    // the next row's values on their way; with fp32 rows and 16 values a lane they would spill
    constexpr bool AHEAD = MULTI && (THREADS == kNormHalf || (THREADS <= 512 && sizeof(W) == 2));
    __shared__ float slots[2][16];
    __shared__ float join[MULTI ? 1 : 2 * 64 * N];
    Team<CH, NC, MULTI> t(p.D);
    Raw<ALL, STREAM, V, CH, NC> raw_o, raw_g, raw_da;
    Raw<ALL, STREAM, W, CH, NC> raw_r, raw_dr;
    const auto fetch = [&](int64_t row) {
        raw_o.load(p.o, p.ldo, row, t);
        raw_g.load(p.gate, p.ldg, row, t);
        raw_r.load(p.res, p.ldres, row, t);
        raw_da.load(p.da, p.ldda, row, t);
        raw_dr.load(p.dr, p.lddr, row, t);
    };
    if (AHEAD && t.row < p.rows) fetch(t.row);
    float kw[N], w2[N], c1[N], c2[N];
    load_weights<true>(kw, w2, p, t);
#pragma unroll
    for (int i = 0; i < N; ++i) c1[i] = c2[i] = 0.f;
    for (; t.row < p.rows; t.row += t.rows_step) {
        float o[N], g[N], r[N], dr[N], da[N];
        if (!AHEAD) fetch(t.row);
        raw_o.get(o);
        raw_g.get(g);
        raw_r.get(r);
        raw_da.get(da);
        raw_dr.get(dr);
        if (AHEAD && t.row + t.rows_step < p.rows) fetch(t.row + t.rows_step);
        const float q = p.post ? p.saved[t.row] : 1.f, n = p.saved[p.rows + t.row];
        float act[N];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            o[i] *= q;                                   // unit o
            float slope = 0.f;
            act[i] = 1.f;
            if (ALL || p.gate) act[i] = act_of(p.act, g[i], slope);
            g[i] = slope;
            r[i] = fmaf(kw[i], o[i] * act[i], r[i]) * n;   // unit r
            c2[i] = fmaf(da[i], r[i], c2[i]);
            da[i] *= w2[i];
            s = fmaf(da[i], r[i], s);
        }
        const float mean2 = ALL || p.da ? t.sum(s, slots) / (float)p.D : 0.f;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dr[i] = fmaf(n, fmaf(-r[i], mean2, da[i]), dr[i]);   // dR
            const float e = dr[i] * act[i];
            c1[i] = fmaf(e, o[i], c1[i]);
            act[i] = e * kw[i];
            s = fmaf(act[i], o[i], s);
        }
        if (p.dres) store_row<TAIL, W>(dr, p.dres, p.lddres, t);
        const float mean1 = p.post && p.d_o ? t.sum(s, slots) / (float)p.D : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] *= dr[i] * kw[i] * o[i];
            o[i] = p.post ? q * fmaf(-o[i], mean1, act[i]) : act[i];
        }
        if (p.dgate) store_row<TAIL, V>(g, p.dgate, p.lddg, t);
        if (p.d_o) store_row<TAIL, V>(o, p.d_o, p.lddo, t);
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
        Chunk<float, CH> s1, s2;
#pragma unroll
        for (int i = 0; i < CH; ++i) s1[i] = c1[j * CH + i], s2[i] = c2[j * CH + i];
        store_chunk<TAIL, float, CH>(part, t.at[j], s1);
        store_chunk<TAIL, float, CH>(part + p.D, t.at[j], s2);
    }
}

// The workgroups' column sums; dw1 and dk are the one sum of dR act o q times k
// and w1.
__global__ void __launch_bounds__(1024) k_norm_columns(NormArgs p, int groups, float *dw1, float *dk, float *dw2) {
    const int i = blockIdx.x * 64 + (threadIdx.x & 63);
    float s;
    if (!column_sum(p.part, p.D, groups, i, s)) return;
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

// Backwards, rows of five or six waves at 16 values a lane leave a CU's eight
// places partly empty and its four SIMDs unevenly loaded: 8 values a lane then, and
// nine to twelve waves of the twelve that their registers allow.  1999 x 5001 fp16
// training 82 -> 75 us, 8888 x 4500 bf16 with fp32 rows 328 -> 291, 6510 x 6144 fp16
// 217 -> 206; below, 13333 x 3000 fp16 195 -> 251, 20000 x 4096 bf16 387 -> 427.
bool half_lanes(int D) { return D > 4096 && D <= 6144; }

// Workgroups: as many as are resident together (16 waves a CU forwards, and
// backwards 8, 16 or 24 with 16, 8 or 4 values a lane, 12 with half_lanes), so that
// a team runs through its rows without a second round of workgroups, and the
// backward pass has few column sums; the rows are spread evenly.  One kind is not
// resident as counted: forwards over fp32 rows of 1025 to 8192 values the registers
// (132 to 158) allow 12 waves, and what is left of the 16 begins as the others end.  Training over rows of 5001 at 16 values a lane in 512 workgroups instead
// of 256: 99 us against 90; of 256 in 512 instead of
// 1024: 200 against 185.  Forwards one wave a row takes twice as many (310 us
// against 316).
unsigned norm_groups(const fi_norm_desc *q, bool backward) {
    const int ch = value_bytes(q->res_dtype) == 2 ? 8 : 4, D = q->channels, waves = team_waves(D);
    const bool half = backward && half_lanes(D);
    const int group = half ? (D + 511) / 512 : waves > 1 ? waves : 4;
    const int resident = half ? 12 : !backward ? 16 : D <= 64 * 4 && ch == 4 ? 24 : D <= 64 * 8 ? 16 : 8;
    const int64_t most = kNormCUs * std::max(1, resident / group) * (!backward && waves == 1 ? 2 : 1);
    const int64_t need = std::max<int64_t>(1, waves > 1 ? q->rows : (q->rows + 3) / 4);
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

template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS, bool TAIL, bool ALL, bool STREAM>
void launch(const NormArgs &a, bool backward, unsigned groups, unsigned threads, hipStream_t st) {
    if (backward)
        hipLaunchKernelGGL((k_norm_back<V, W, CH, NC, MULTI, TAIL, ALL, STREAM, THREADS>), dim3(groups), dim3(threads), 0,
                           st, a);
    else if constexpr (THREADS != kNormHalf)
        hipLaunchKernelGGL((k_norm<V, W, CH, NC, MULTI, TAIL, ALL, STREAM, THREADS>), dim3(groups), dim3(threads), 0, st,
                           a);
}

// With every tensor of a row given, without (and always at the smallest and
// widest rows) the kernels that check for each.  Inputs of more than the
// last-level cache are read as streams: 131072 x 864 rows 302 -> 293 us, a
// training pass 695 -> 666; below that a producer's output may still be cached,
// and reading it so costs (a chain of scan, norm, scan over 4096 x 864 38.4
// against 35.6 us).
template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS>
void launch(const NormArgs &a, bool backward, unsigned groups, unsigned threads, hipStream_t st) {
    const bool all = a.o && a.gate && a.res && (!backward || (a.dr && a.da));
    const int64_t values = a.rows * a.D;
    const bool stream = values * (int64_t)((backward ? 3 : 2) * sizeof(V) + (backward ? 2 : 1) * sizeof(W)) > kNormCache;
    if constexpr (CH > 1 && THREADS <= kNormHalf) {
        if (all && a.D % CH == 0) {
            if (stream) return launch<V, W, CH, NC, MULTI, THREADS, false, true, true>(a, backward, groups, threads, st);
            return launch<V, W, CH, NC, MULTI, THREADS, false, true, false>(a, backward, groups, threads, st);
        }
        if (all) {
            if (stream) return launch<V, W, CH, NC, MULTI, THREADS, true, true, true>(a, backward, groups, threads, st);
            return launch<V, W, CH, NC, MULTI, THREADS, true, true, false>(a, backward, groups, threads, st);
        }
    }
    launch<V, W, CH, NC, MULTI, THREADS, true, false, false>(a, backward, groups, threads, st);
}

template <typename V, typename W>
void launch(const NormArgs &a, bool backward, unsigned groups, hipStream_t st) {
    constexpr int CH = sizeof(W) == 2 ? 8 : 4;
    const int waves = team_waves(a.D);
    if (backward && half_lanes(a.D))
        launch<V, W, CH, kRowLane / 2 / CH, true, kNormHalf>(a, backward, groups, (a.D + 511) / 512 * 64, st);
    else if (a.D < CH)
        launch<V, W, 1, 1, false, 256>(a, backward, groups, 256, st);
    else if (a.D <= 64 * CH)
        launch<V, W, CH, 1, false, 256>(a, backward, groups, 256, st);
    else if (a.D <= 128 * CH)
        launch<V, W, CH, 2, false, 256>(a, backward, groups, 256, st);
    else if (waves == 1)
        launch<V, W, CH, kRowLane / CH, false, 256>(a, backward, groups, 256, st);
    else if (waves <= 8)
        launch<V, W, CH, kRowLane / CH, true, 512>(a, backward, groups, waves * 64, st);
    else
        launch<V, W, CH, kRowLane / CH, true, 1024>(a, backward, groups, waves * 64, st);
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
    return up256((size_t)norm_groups(desc, true) * 2 * desc->channels * sizeof(float));
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
    if (!aligned(es, {o, gate, a}) || !aligned(rs, {res, r}) || !aligned(4, {post_weight, scale, pre_weight, saved}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const View vr = {r, n.rows, D * rs, n.ldr * rs}, vres = {res, n.rows, D * rs, n.ldres * rs};
    const View out[] = {vr, {a, n.rows, D * es, n.lda * es}, {saved, 1, (size_t)n.rows * 8, (size_t)n.rows * 8}};
    const View in[] = {{o, n.rows, D * es, n.ldo * es}, {gate, n.rows, D * es, n.ldg * es},
                       {post_weight, 1, D * 4, D * 4}, {scale, 1, D * 4, D * 4}, {pre_weight, 1, D * 4, D * 4}};
    const bool inplace = same_view(vr, vres);
    if (outputs_meet(out, 3, in, 5) || outputs_meet(out + 1, 2, &vres, 1) || (!inplace && views_meet(vr, vres)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    n.o = o, n.gate = gate, n.res = res, n.w1 = post_weight, n.k = scale, n.w2 = pre_weight;
    n.r = r, n.a = a, n.saved = saved;
    launch(desc, n, false, norm_groups(desc, false), (hipStream_t)stream);
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
    if (!aligned(es, {o, gate, da, d_o, dgate}) || !aligned(rs, {res, dr, dres}) ||
        !aligned(4, {post_weight, scale, pre_weight, saved, dpost, dscale, dpre}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
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
    const unsigned groups = n.rows > 0 ? norm_groups(desc, true) : 0;
    if (groups) launch(desc, n, true, groups, st);
    if (n.columns)
        hipLaunchKernelGGL(k_norm_columns, dim3((unsigned)((2 * D + 63) / 64)), dim3(1024), 0, st, n, (int)groups, dpost, dscale, dpre);
    return op_launched(call);
}

}  // extern "C"
