// The layer norm with a residual and its gradients (fi_layer_*).  Per row of D
// values:
//   r = res + x;  u = (r - m) p, m = mean r, p = 1/sqrt(mean (r - m)^2 + eps);
//   a = u w + b.
// Backwards, with e = da w:
//   dR = dr + p (e - mean(e) - u mean(e u)),  dx = dres = dR,
//   dw = sum da u,  db = sum da   (over the rows).
// r is formed again from x and res in fp32, not read back rounded.
#include "fi_rows.h"

namespace fi {

namespace {

constexpr int kLayerMaxD = 16384;
constexpr int64_t kLayerCache = 256 << 20;   // bytes of the last-level cache
constexpr int kLayerCUs = 256;         // compute units that the workgroups are spread over

struct LayerArgs {
    const void *x, *res, *dr, *da;
    void *r, *a, *dx, *dres;
    const float *w, *b;
    float *saved;            // [2][rows]: mean, 1/deviation
    float *part;             // [groups][2][D] column sums of da u and of da
    int64_t rows;
    int64_t ldx, ldres, ldr, lda, lddr, ldda, lddx, lddres;
    int D;
    float eps;
    bool columns;            // column sums wanted
};

// A lane's column values of p, `none` where p is null or the lane owns nothing.
template <int CH, int NC, bool MULTI>
__device__ __forceinline__ void load_columns(float (&v)[NC * CH], const float *p, float none, bool owned,
                                             const Team<CH, NC, MULTI> &t) {
    Chunk<float, CH> raw[NC];
    if (p) {
#pragma unroll
        for (int j = 0; j < NC; ++j) raw[j] = load_chunk<float, CH>(p, t.at[j]);
    }
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const float x = p ? raw[j][i] : none;
            v[j * CH + i] = owned && i < t.at[j].skip ? 0.f : x;
        }
}

// Forward: a row in registers, every tensor once.  The mean m0 of the fp32 sum is
// off by its rounding; the mean d of what is left, found along with the squares,
// takes that away (variance mean c^2 - d^2 of c = r - m0), so rows far from zero
// keep their digits.  HBM-bound: 131072 x 864 bf16 with fp32 rows 247 us (5.5 TB/s);
// 1999 x 5001 fp16 without a residual 15 us: few rows, two barriers in each.
template <typename V, typename W, int CH, int NC, bool MULTI, bool TAIL, bool ALL, bool STREAM, int THREADS>
__global__ void __launch_bounds__(THREADS) k_layer(LayerArgs p) {
    constexpr int N = CH * NC;
    constexpr bool AHEAD = MULTI && THREADS <= 512;
    __shared__ float slots[2][2][16];
    Team<CH, NC, MULTI> t(p.D);
    Raw<ALL, STREAM, V, CH, NC> raw_x;
    Raw<ALL, STREAM, W, CH, NC> raw_r;
    const auto fetch = [&](int64_t row) {
        raw_x.load(p.x, p.ldx, row, t);
        raw_r.load(p.res, p.ldres, row, t);
    };
    if (AHEAD && t.row < p.rows) fetch(t.row);
    float w[N], b[N];
    load_columns(w, p.w, 1.f, false, t);
    load_columns(b, p.b, 0.f, false, t);
    const float per = 1.f / (float)p.D;
    for (; t.row < p.rows; t.row += t.rows_step) {
        float x[N], r[N];
        if (!AHEAD) fetch(t.row);
        raw_x.get(x);
        raw_r.get(r);
        if (AHEAD && t.row + t.rows_step < p.rows) fetch(t.row + t.rows_step);
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float c = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                r[j * CH + i] += x[j * CH + i];
                c += TAIL && i < t.at[j].skip ? 0.f : r[j * CH + i];
            }
            s += t.at[j].skip < CH ? c : 0.f;
        }
        if (p.r) store_row<TAIL, W>(r, p.r, p.ldr, t);
        t.sums(s, q, slots);
        const float mean = s * per;
        s = q = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float c = 0.f, e = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                r[j * CH + i] -= mean;
                const float v = TAIL && i < t.at[j].skip ? 0.f : r[j * CH + i];
                c += v;
                e = fmaf(v, v, e);
            }
            s += t.at[j].skip < CH ? c : 0.f;
            q += t.at[j].skip < CH ? e : 0.f;
        }
        t.sums(s, q, slots);
        const float d = s * per;
        const float n = 1.f / sqrtf(fmaxf(fmaf(-d, d, q * per), 0.f) + p.eps);
        if (p.a) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = fmaf((r[i] - d) * n, w[i], b[i]);
            store_row<TAIL, V>(r, p.a, p.lda, t);
        }
        if (p.saved && t.first) {
            p.saved[t.row] = mean + d;
            p.saved[p.rows + t.row] = n;
        }
    }
}

// Backward: every tensor of the row once, its three means in one step: those of e and e u,
// and that of r - m, which takes the rounding of the mean as it is kept away; the column
// sums of a team's rows in registers, its workgroup's joined in LDS (team after
// team, so the order is fixed) and written once.  Elements that a lane does not
// own have weights of zero, so both means pass them by.  131072 x 768 bf16 with fp32
// rows 308 us (5.9 TB/s); 1999 x 5001 fp16 23 us and 6 for the column sums.
template <typename V, typename W, int CH, int NC, bool MULTI, bool TAIL, bool ALL, bool STREAM, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 512 ? 2 : 1) k_layer_back(LayerArgs p) {
    constexpr int N = CH * NC;
    constexpr bool AHEAD = MULTI && THREADS <= 512;
    __shared__ float slots[2][3][16];
    __shared__ float join[MULTI ? 1 : 2 * 64 * N];
    Team<CH, NC, MULTI> t(p.D);
    Raw<ALL, STREAM, V, CH, NC> raw_x, raw_da;
    Raw<ALL, STREAM, W, CH, NC> raw_r, raw_dr;
    const auto fetch = [&](int64_t row) {
        raw_x.load(p.x, p.ldx, row, t);
        raw_r.load(p.res, p.ldres, row, t);
        raw_da.load(p.da, p.ldda, row, t);
        raw_dr.load(p.dr, p.lddr, row, t);
    };
    if (AHEAD && t.row < p.rows) fetch(t.row);
    float w[N], c1[N], c2[N];
    load_columns(w, p.w, 1.f, true, t);
#pragma unroll
    for (int i = 0; i < N; ++i) c1[i] = c2[i] = 0.f;
    const float per = 1.f / (float)p.D;
    for (; t.row < p.rows; t.row += t.rows_step) {
        float x[N], r[N], dr[N], da[N];
        if (!AHEAD) fetch(t.row);
        raw_x.get(x);
        raw_r.get(r);
        raw_da.get(da);
        raw_dr.get(dr);
        if (AHEAD && t.row + t.rows_step < p.rows) fetch(t.row + t.rows_step);
        const float mean = p.saved[t.row], n = p.saved[p.rows + t.row];
        float s = 0.f, q = 0.f, d = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float c = 0.f, e = 0.f, m = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int at = j * CH + i;
                r[at] = r[at] + x[at] - mean;
                m += TAIL && i < t.at[j].skip ? 0.f : r[at];
                const float g = da[at] * w[at];
                c += g;
                e = fmaf(g, r[at], e);
            }
            s += t.at[j].skip < CH ? c : 0.f;
            q += t.at[j].skip < CH ? e : 0.f;
            d += t.at[j].skip < CH ? m : 0.f;
        }
        t.sums(s, q, d, slots);
        s *= per, d *= per;
        q = n * fmaf(-d, s, q * per);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float u = (r[i] - d) * n;                  // unit r
            c1[i] = fmaf(da[i], u, c1[i]);
            c2[i] += da[i];
            dr[i] = fmaf(n, fmaf(da[i], w[i], -fmaf(u, q, s)), dr[i]);
        }
        if (p.dres) store_row<TAIL, W>(dr, p.dres, p.lddres, t);
        if (p.dx) store_row<TAIL, V>(dr, p.dx, p.lddx, t);
    }
    if (!p.columns) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
    if (!MULTI) {
        for (int k = 0; k < t.waves; ++k) {
            if (t.wave == k) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = i * 64 + t.lane;
                    if (k) c1[i] += join[at], c2[i] += join[64 * N + at];
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

__global__ void __launch_bounds__(1024) k_layer_columns(LayerArgs p, int groups, float *dw, float *db) {
    const int i = blockIdx.x * 64 + (threadIdx.x & 63);
    float s;
    if (!column_sum(p.part, p.D, groups, i, s)) return;
    if (i >= p.D) {
        if (db) db[i - p.D] = s;
    } else if (dw)
        dw[i] = s;
}

const char *layer_check(const fi_layer_desc *q) {
    if (!q) return "null descriptor";
    if (q->rows < 0 || q->rows > (int64_t(1) << 40)) return "rows is negative or over 2^40";
    if (q->channels < 1 || q->channels > kLayerMaxD) return "channels is not in 1 .. 16384";
    if (!value_type(q->dtype)) return "dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->res_dtype != q->dtype && q->res_dtype != FI_F32) return "res_dtype is neither dtype nor FI_F32";
    if (!(q->eps >= 0.f)) return "eps is negative or not a number";
    const int64_t ld[] = {q->ld_x, q->ld_res, q->ld_r, q->ld_a, q->ld_dr, q->ld_da, q->ld_dx, q->ld_dres};
    for (int64_t v : ld)
        if (v != 0 && (v < q->channels || v > (int64_t(1) << 40))) return "a row pitch is less than channels";
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    return nullptr;
}

// Workgroups: as many as are resident together, so that a team runs through its
// rows without a second round of workgroups, and the backward pass has few column
// sums; the rows are spread evenly.  The counts are those of the block's norms, whose
// rows lie in registers alike.
unsigned layer_groups(const fi_layer_desc *q, bool backward) {
    const int D = q->channels, waves = team_waves(D), ch = value_bytes(q->res_dtype) == 2 ? 8 : 4;
    const int group = waves > 1 ? waves : 4;
    const int resident = !backward ? 16 : D <= 64 * 4 && ch == 4 ? 24 : D <= 64 * 8 ? 16 : 8;
    const int64_t most = kLayerCUs * std::max(1, resident / group) * (!backward && waves == 1 ? 2 : 1);
    const int64_t need = std::max<int64_t>(1, waves > 1 ? q->rows : (q->rows + 3) / 4);
    const int64_t turns = (need + most - 1) / most;
    return (unsigned)((need + turns - 1) / turns);
}

void layer_args(const fi_layer_desc *q, LayerArgs &a) {
    a.rows = q->rows;
    a.D = q->channels;
    a.eps = q->eps;
    a.ldx = pitch_or(q->ld_x, a.D);
    a.ldres = pitch_or(q->ld_res, a.D);
    a.ldr = pitch_or(q->ld_r, a.D);
    a.lda = pitch_or(q->ld_a, a.D);
    a.lddr = pitch_or(q->ld_dr, a.D);
    a.ldda = pitch_or(q->ld_da, a.D);
    a.lddx = pitch_or(q->ld_dx, a.D);
    a.lddres = pitch_or(q->ld_dres, a.D);
}

template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS, bool TAIL, bool ALL, bool STREAM>
void launch(const LayerArgs &a, bool backward, unsigned groups, unsigned threads, hipStream_t st) {
    if (backward)
        hipLaunchKernelGGL((k_layer_back<V, W, CH, NC, MULTI, TAIL, ALL, STREAM, THREADS>), dim3(groups), dim3(threads),
                           0, st, a);
    else
        hipLaunchKernelGGL((k_layer<V, W, CH, NC, MULTI, TAIL, ALL, STREAM, THREADS>), dim3(groups), dim3(threads), 0,
                           st, a);
}

// With every tensor of a row given, without (and always at the smallest and
// widest rows) the kernels that check for each.  Inputs of more than the
// last-level cache are read as streams.
template <typename V, typename W, int CH, int NC, bool MULTI, int THREADS>
void launch(const LayerArgs &a, bool backward, unsigned groups, unsigned threads, hipStream_t st) {
    const bool all = a.x && a.res && (!backward || (a.dr && a.da));
    const int64_t values = a.rows * a.D;
    const bool stream = values * (int64_t)((backward ? 2 : 1) * (sizeof(V) + sizeof(W))) > kLayerCache;
    if constexpr (CH > 1 && THREADS <= 512) {
        if (all && a.D % CH == 0) {
            if (stream) return launch<V, W, CH, NC, MULTI, THREADS, false, true, true>(a, backward, groups, threads, st);
            return launch<V, W, CH, NC, MULTI, THREADS, false, true, false>(a, backward, groups, threads, st);
        }
    }
    launch<V, W, CH, NC, MULTI, THREADS, true, false, false>(a, backward, groups, threads, st);
}

template <typename V, typename W>
void launch(const LayerArgs &a, bool backward, unsigned groups, hipStream_t st) {
    constexpr int CH = sizeof(W) == 2 ? 8 : 4;
    const int waves = team_waves(a.D);
    if (a.D < CH)
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

void launch(const fi_layer_desc *q, const LayerArgs &a, bool backward, unsigned groups, hipStream_t st) {
    if (q->dtype == FI_F32) launch<float, float>(a, backward, groups, st);
    else if (q->dtype == FI_BF16)
        q->res_dtype == FI_F32 ? launch<bf16_t, float>(a, backward, groups, st)
                               : launch<bf16_t, bf16_t>(a, backward, groups, st);
    else
        q->res_dtype == FI_F32 ? launch<f16_t, float>(a, backward, groups, st)
                               : launch<f16_t, f16_t>(a, backward, groups, st);
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_layer_workspace_bytes(const fi_layer_desc *desc) {
    if (layer_check(desc)) return 0;
    return up256((size_t)layer_groups(desc, true) * 2 * desc->channels * sizeof(float));
}

fi_status fi_layer_forward(const fi_layer_desc *desc, const void *x, const void *res, const float *weight,
                           const float *bias, void *r, void *a, float *saved, void *stream) {
    static const char *call = "fi_layer_forward";
    if (const char *why = layer_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (desc->rows == 0 || (!r && !a && !saved)) return FI_OK;
    if (!x && !res) return op_fail(FI_EINVAL, call, "x or res is required");
    LayerArgs n = {};
    layer_args(desc, n);
    const size_t es = value_bytes(desc->dtype), rs = value_bytes(desc->res_dtype), D = n.D;
    if (!aligned(es, {x, a}) || !aligned(rs, {res, r}) || !aligned(4, {weight, bias, saved}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const View vr = {r, n.rows, D * rs, n.ldr * rs}, vres = {res, n.rows, D * rs, n.ldres * rs};
    const View out[] = {vr, {a, n.rows, D * es, n.lda * es}, {saved, 1, (size_t)n.rows * 8, (size_t)n.rows * 8}};
    const View in[] = {{x, n.rows, D * es, n.ldx * es}, {weight, 1, D * 4, D * 4}, {bias, 1, D * 4, D * 4}};
    const bool inplace = same_view(vr, vres);
    if (outputs_meet(out, 3, in, 3) || outputs_meet(out + 1, 2, &vres, 1) || (!inplace && views_meet(vr, vres)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    n.x = x, n.res = res, n.w = weight, n.b = bias;
    n.r = r, n.a = a, n.saved = saved;
    launch(desc, n, false, layer_groups(desc, false), (hipStream_t)stream);
    return op_launched(call);
}

fi_status fi_layer_backward(const fi_layer_desc *desc, const void *x, const void *res, const float *weight,
                            const float *saved, const void *dr, const void *da, void *dx, void *dres, float *dweight,
                            float *dbias, void *workspace, void *stream) {
    static const char *call = "fi_layer_backward";
    if (const char *why = layer_check(desc)) return op_fail(FI_EINVAL, call, why);
    LayerArgs n = {};
    layer_args(desc, n);
    if (n.rows > 0) {
        if (!x && !res) return op_fail(FI_EINVAL, call, "x or res is required");
        if (!saved || !workspace || (uintptr_t)workspace % 256)
            return op_fail(FI_EINVAL, call, "saved and a workspace aligned to 256 bytes are required");
        if ((dx && !x) || (dres && !res) || ((dweight || dbias) && !da))
            return op_fail(FI_EINVAL, call, "a gradient is asked for whose input is not given");
    }
    const size_t es = value_bytes(desc->dtype), rs = value_bytes(desc->res_dtype), D = n.D;
    if (!aligned(es, {x, da, dx}) || !aligned(rs, {res, dr, dres}) || !aligned(4, {weight, saved, dweight, dbias}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const size_t ws = fi_layer_workspace_bytes(desc);
    const View vdr = {dr, n.rows, D * rs, n.lddr * rs}, vdres = {dres, n.rows, D * rs, n.lddres * rs};
    const View out[] = {vdres, {dx, n.rows, D * es, n.lddx * es}, {dweight, 1, D * 4, D * 4}, {dbias, 1, D * 4, D * 4},
                        {workspace, 1, ws, ws}};
    const View in[] = {{x, n.rows, D * es, n.ldx * es}, {res, n.rows, D * rs, n.ldres * rs},
                       {da, n.rows, D * es, n.ldda * es}, {weight, 1, D * 4, D * 4},
                       {saved, 1, (size_t)n.rows * 8, (size_t)n.rows * 8}};
    const bool inplace = same_view(vdr, vdres);
    if (outputs_meet(out, 5, in, 5) || outputs_meet(out + 1, 4, &vdr, 1) || (!inplace && views_meet(vdr, vdres)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    n.x = x, n.res = res, n.w = weight;
    n.saved = (float *)saved, n.dr = dr, n.da = da, n.dx = dx, n.dres = dres;
    n.part = (float *)workspace, n.columns = dweight || dbias;
    const hipStream_t st = (hipStream_t)stream;
    const unsigned groups = n.rows > 0 ? layer_groups(desc, true) : 0;
    if (groups && (dx || dres || n.columns)) launch(desc, n, true, groups, st);
    if (n.columns)
        hipLaunchKernelGGL(k_layer_columns, dim3((unsigned)((2 * D + 63) / 64)), dim3(1024), 0, st, n, (int)groups,
                           dweight, dbias);
    return op_launched(call);
}

}  // extern "C"
