// The gated delta rule's gradients.  Per chunk, with D the gradient of the state
// behind it, w and S as the forward pass kept them, N = (I + A')^-1,
// A'_ij = b_i E_ij (k_i . k_j) (i > j) and dy scaled:
//   x = N^T (P^T dy + e^(G_C - G) K D),  dv = b x,  dbeta_i = x_i . w_i,
//   the gradient before it  e^(G_C) D + (e^G Q)^T dy - (e^G K)^T dv,
// which again passes from chunk to chunk column by column, from the last to the
// first.  The rest is a chunk's own, with H_ij = -b_i b_j E_ij (x_i . w_j) (i > j) and
// J_ij = b_j E_ij (dy_i . w_j) (i >= j):
//   dq_i = sum_j J_ij k_j + e^G_i S dy_i,
//   dk_i = sum_j (H_ij + H_ji) k_j + sum_j J_ji q_j - e^G_i S dv_i + e^(G_C - G_i) b_i D w_i,
//   ddecay_t = e^(G_C) <D, S> + sum_{i >= t > j} (H_ij k_i . k_j + J_ij q_i . k_j)
//            + sum_{i >= t} e^G_i (q_i . S dy_i - k_i . S dv_i) + sum_{j < t} e^(G_C - G_j) b_j k_j . D w_j.
// A decay scales what was before it against what comes after: each of its four parts
// holds only terms that carry it, so a gate that is nearly shut keeps the digits of its
// gradient.  (<D, S'> + sum_{i >= t} (q_i . dq_i - v_i . dv_i) is the same number, but as
// a difference of others that do not carry the decay.)
#include "fi_delta.h"

namespace fi {

namespace {

// The gradient of the state through a segment's chunks, 16 columns a wave, backwards.
// FULL: from the gradient behind the segment; dv, x and the gradients behind each
// chunk.  Else from nothing, only the gradient before the segment.  Loads as in the
// forward pass, but those of q and dy begin with their chunk: ahead of it they would
// spill (205 us against 368 in a training pass over 8192 x 4 x 6 heads of 128); q's
// transpose takes the place of k in LDS after k's last use.
template <typename T, int KT, bool FULL>
__global__ void __launch_bounds__(512, 4) k_delta_back_chain(DeltaArgs p) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms;
    constexpr int MT = C / 16, CS = C / 32, DT = KT * 2, DK = KT * 32;
    constexpr int KB = C * DK * 2, MB = tri_pieces<C>() * kPiece;
    extern __shared__ __align__(16) char lds[];
    char *const ik = lds, *const iqt = lds, *const ikt = ik + N * KB, *const in = ikt + N * KB, *const ip = in + 3 * MB;
    char *const ff = ip + 3 * MB;
    const float *const f = reinterpret_cast<const float *>(ff);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.B * p.H, seg = blockIdx.x / heads + (FULL ? 0 : 1), bh = blockIdx.x % heads, b = bh / p.H, h = bh % p.H;
    const int column = (blockIdx.y * (int)(blockDim.x >> 6) + wave) * 16 + (lane & 15);
    const bool mine = column < p.dv;
    const int64_t length = delta_length(p, b), size = (int64_t)p.dk * p.dv;
    const int hk = h / (p.H / p.HK);

    f32x4 D[DT];
    const float *from = !FULL ? nullptr : p.segments > 1 ? p.starts + ((int64_t)seg * heads + bh) * size
                                        : p.dfinal       ? p.dfinal + bh * size
                                                         : nullptr;
#pragma unroll
    for (int t = 0; t < DT; ++t) D[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (from) load_state(D, from, p.dk, p.dv, column);
    const T *const q = static_cast<const T *>(p.q) + hk * p.dk, *const k = static_cast<const T *>(p.k) + hk * p.dk;
    const T *const dy = static_cast<const T *>(p.dy) + (int64_t)h * p.dv;
    T *const dv = FULL ? static_cast<T *>(p.dv_out) + (int64_t)h * p.dv : nullptr;
    const int64_t first = seg * p.per, last = min(p.chunks, first + p.per);
    const int64_t stop = min(last, (length + C - 1) / C);
    if (FULL && mine)
        for (int64_t c = max(first, stop); c < last; ++c) {
            const int rows = (int)min<int64_t>(C, p.T - c * C);
            for (int i = lane >> 4; i < rows; i += 4) dv[((c * C + i) * p.B + b) * p.lddv + column] = (T)0.f;
        }
    Stage<T, C, DK, true> sk, sq;
    T ys[MT][4];
    const auto rows_from = [&](const T *x, int64_t ld, int64_t c) { return x + (c * C * p.B + b) * ld; };
    const auto live_of = [&](int64_t c) { return (int)min<int64_t>(C, length - c * C); };
    const auto ahead = [&](int64_t c) { sk.load(rows_from(k, p.ldk, c), (unsigned)(p.B * p.ldk), p.dk, live_of(c)); };
    const auto matrices = [&](int64_t c) {                    // N, P and the factors
        const int64_t at = c * heads + bh;
        bring(in, p.images + at * image_bytes<T>(), 6 * MB);
        bring(ff, (const char *)(p.factors + at * kDeltaFactors * C), factor_bytes<C>());
    };
    if (first < stop) ahead(stop - 1), matrices(stop - 1);
    for (int64_t c = stop - 1; c >= first; --c) {
        const int64_t t0 = c * C, at = c * heads + bh;
        const int rows = (int)min<int64_t>(C, p.T - t0), live = live_of(c);
        __syncthreads();
        sk.put(p.dk, live, ik, ikt);
        __syncthreads();
        load_column<T, MT>(ys, rows_from(dy, p.lddy, c), min(column, p.dv - 1), (unsigned)(p.B * p.lddy), live);
        sq.load(rows_from(q, p.ldq, c), (unsigned)(p.B * p.ldq), p.dk, live);
        if (FULL) store_state(p.ends + at * size, D, p.dk, p.dv, column);
        f32x4 X[MT], Y[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) X[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KT; ++ks) {
            const Frag<3> s = step_of<3>(D, ks);
#pragma unroll
            for (int i = 0; i < MT; ++i) multiply<2>(X[i], piece<N>(ik, i * KT + ks, KB), s);
            in_order();
        }
        arrived();
        __syncthreads();
        const int ylive = anew(live);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + tile_row(r);
                X[i][r] *= f[row];
                Y[i][r] = row < ylive ? (float)ys[i][r] : 0.f;
            }
        sq.put(p.dk, live, nullptr, iqt);
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            const Frag<N> s = step_of<N>(Y, cs);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                if (tri_in<C, true>(i, cs)) multiply<2>(X[i], piece<3>(ip, tri_at<C, true>(i, cs), MB), s);
            in_order();
        }
        f32x4 Z[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) Z[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            const Frag<3> s = step_of<3>(X, cs);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                if (tri_in<C, true>(i, cs)) multiply<2>(Z[i], piece<3>(in, tri_at<C, true>(i, cs), MB), s);
            in_order();
        }
        if (c > first) ahead(c - 1);
        if (FULL && mine) {
            store_column<float, MT>(p.x + at * C * p.dv, column, p.dv, Z, C, C);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) X[i][r] = Z[i][r] * f[3 * C + i * 16 + tile_row(r)];
            store_column<T, MT>(dv + (t0 * p.B + b) * p.lddv, column, (unsigned)(p.B * p.lddv), X, rows, live);
        }
        const float decay = f[4 * C];
#pragma unroll
        for (int t = 0; t < DT; ++t) D[t] *= decay;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + tile_row(r);
                Y[i][r] *= f[C + row];
                Z[i][r] *= -f[2 * C + row];
            }
        __syncthreads();
        if (c > first) matrices(c - 1);
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            const Frag<3> sy = step_of<3>(Y, cs);
#pragma unroll
            for (int t = 0; t < DT; ++t) multiply<2>(D[t], piece<N>(iqt, t * CS + cs, KB), sy);
            in_order();
            const Frag<3> sz = step_of<3>(Z, cs);
#pragma unroll
            for (int t = 0; t < DT; ++t) multiply<2>(D[t], piece<N>(ikt, t * CS + cs, KB), sz);
            in_order();
        }
    }
    if (!FULL)
        store_state(p.local + ((int64_t)seg * heads + bh) * size, D, p.dk, p.dv, column);
    else if (seg == 0 && p.dstate)
        store_state(p.dstate + bh * size, D, p.dk, p.dv, column);
}

// Sums over the lanes up to each one of a half (32 lanes): shifts within rows of 16
// lanes, then the lower row's last lane into the upper row.
__device__ __forceinline__ float half_sums(float v) {
#define FI_LANE_ADD(ctrl, rows) \
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false))
    FI_LANE_ADD(0x111, 0xf);
    FI_LANE_ADD(0x112, 0xf);
    FI_LANE_ADD(0x114, 0xf);
    FI_LANE_ADD(0x118, 0xf);
    FI_LANE_ADD(0x142, 0xa);
#undef FI_LANE_ADD
    return v;
}

// What is a chunk's own, for a key head and the heads that share it: a workgroup a
// chunk, a wave 32 channels of the keys.  The values' channels pass in slabs of 32; H
// and J then take the slabs' place in LDS, so that two workgroups share a CU and one
// computes while the other waits for its slab (one workgroup where heads share a key
// head: SHARED, their sums take 64 registers more).  The decays' pairs of positions are
// multiplied out there, with k and q read again (as images by rows they would leave a CU
// one workgroup): 85 us of it.  8192 x 4 x 6 heads of 128 bf16 560 us (0.5 GB: 100 at a
// copy's rate): 92 registers spill, a slab's two barriers and its loads of the states.
// The steps of k and q by twos ahead of their products 559, by fours 680.
template <typename T, int KT, bool VEC, bool SHARED>
__global__ void __launch_bounds__(256, SHARED ? 1 : 2) k_delta_grads(DeltaArgs p) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms;
    constexpr int MT = C / 32, CS = C / 16, DK = KT * 32, KB = C * DK * 2, LD = C + 4, SB = MT * 2 * kPiece;
    extern __shared__ __align__(16) char lds[];
    char *const ikt = lds, *const iqt = ikt + N * KB, *const ix = iqt + N * KB, *const iw = ix + 3 * SB, *const iy = iw + 3 * SB;
    float *const Hm = reinterpret_cast<float *>(ix), *const Jm = Hm + C * LD;
    __shared__ double G[C];
    __shared__ float beta[C], rk[C], rq[C], dotb[C], dots[4][C], dote[4][C], pairs[2][C], total[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5, col = lane & 31;
    const int hk = blockIdx.x % p.HK, b = blockIdx.x / p.HK % p.B, share = p.H / p.HK, heads = p.B * p.H;
    const int64_t c = blockIdx.x / p.HK / p.B, t0 = c * C, n = delta_length(p, b) - t0;
    const int rows = (int)min<int64_t>(C, p.T - t0), live = n < 0 ? 0 : n < rows ? (int)n : rows;
    T *const dq = static_cast<T *>(p.dq) + hk * p.dk, *const dk = static_cast<T *>(p.dk_out) + hk * p.dk;
    if (live == 0) {
        for (int u = tid; u < rows * p.dk; u += 256) {
            const int64_t row = (t0 + u / p.dk) * p.B + b;
            dq[row * p.lddq + u % p.dk] = (T)0.f;
            dk[row * p.lddk + u % p.dk] = (T)0.f;
        }
        for (int u = tid; u < rows * share; u += 256) {
            const int64_t row = (t0 + u / share) * p.B + b;
            p.dg[row * p.lddg + hk * share + u % share] = 0.f;
            p.dbeta[row * p.lddb + hk * share + u % share] = 0.f;
        }
        return;
    }
    const int64_t row0 = t0 * p.B + b;
    {
        Stage<T, C, DK, false> sk, sq;
        sk.load(static_cast<const T *>(p.k) + hk * p.dk + row0 * p.ldk, (unsigned)(p.B * p.ldk), p.dk, live);
        sq.load(static_cast<const T *>(p.q) + hk * p.dk + row0 * p.ldq, (unsigned)(p.B * p.ldq), p.dk, live);
        sk.put(p.dk, live, nullptr, ikt);
        sq.put(p.dk, live, nullptr, iqt);
    }
    // four positions of this lane's channel, of an image of k or q
    const auto four = [&](const char *image, int i, float (&x)[4]) {
        x[0] = x[1] = x[2] = x[3] = 0.f;
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const bf16x4 v = *reinterpret_cast<const bf16x4 *>(image + t * KB + image_at(wave * 32 + col, i, CS));
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += (float)v[j];
        }
    };
    const int d = wave * 32 + col;                       // this lane's channel
    f32x16 ys[MT], xs[MT], sums[2][SHARED ? MT : 1];
    f32x16 *const allq = SHARED ? sums[0] : ys, *const allk = SHARED ? sums[1] : xs;
#pragma unroll
    for (int i = 0; i < (SHARED ? MT : 1); ++i) sums[0][i] = sums[1][i] = zeros16();
    // kk_ij = k_i . k_j and qk_ij = q_i . k_j of a 32 x 32 block, rows i of block a
    const auto products = [&](f32x16 &kk, f32x16 &qk, int a, int b32, auto vec) {
        constexpr bool V = decltype(vec)::value;
        const T *const k0 = static_cast<const T *>(p.k) + hk * p.dk + row0 * p.ldk;
        const T *const q0 = static_cast<const T *>(p.q) + hk * p.dk + row0 * p.ldq;
        const auto operand = [&](const T *from, int64_t ld, int i, int ks) {
            float lo[4], hi[4], x[8];
            const T *row = from + (int64_t)min(i, live - 1) * p.B * ld;
            load4<V>(lo, row, ks * 16 + 4 * half, p.dk, i < live);
            load4<V>(hi, row, ks * 16 + 4 * half + 8, p.dk, i < live);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = lo[j], x[4 + j] = hi[j];
            return split<N>(x);
        };
#pragma unroll 1
        for (int ks = 0; ks < KT * 2; ++ks) {
            const Frag<N> kb = operand(k0, p.ldk, b32 * 32 + col, ks);
            multiply<2>(kk, operand(k0, p.ldk, a * 32 + col, ks), kb);
            multiply<2>(qk, operand(q0, p.ldq, a * 32 + col, ks), kb);
        }
    };

    for (int s = 0; s < share; ++s) {
        const int h = hk * share + s;
        const int64_t at = c * heads + b * p.H + h;
        __syncthreads();
        if (tid < C) {
            const float *f = p.factors + at * kDeltaFactors * C;
            beta[tid] = f[3 * C + tid], rk[tid] = f[5 * C + tid], rq[tid] = f[6 * C + tid];
            G[tid] = (double)f[7 * C + tid] + (double)f[8 * C + tid];
        }
        const float *const x = p.x + at * C * p.dv, *const w = p.w + at * C * p.dv;
        const float *const S = p.states + at * p.dk * p.dv, *const D = p.ends + at * p.dk * p.dv;
        const T *const dy = static_cast<const T *>(p.dy) + row0 * p.lddy + (int64_t)h * p.dv;
        f32x16 wd[MT], xw = zeros16(), yw = zeros16();
#pragma unroll
        for (int i = 0; i < MT; ++i) ys[i] = xs[i] = wd[i] = zeros16();
        float db[MT], inner = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) db[i] = 0.f;
        Chunk<float, 4> na[MT], nu[MT];
        Chunk<T, 4> ny[MT];
        const auto load = [&](int c0) {
#pragma unroll
            for (int e = 0; e < MT; ++e) {
                const int cc = c0 + tid % 8 * 4;
                const int64_t i = min(e * 32 + tid / 8, live - 1);
                na[e] = raw4<VEC>(x + i * p.dv, cc, p.dv);
                nu[e] = raw4<VEC>(w + i * p.dv, cc, p.dv);
                ny[e] = raw4<VEC>(dy + i * p.B * p.lddy, cc, p.dv);
            }
        };
        for (int c0 = 0; c0 < p.dv; c0 += 32) {
            load(c0);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < MT; ++e) {
                const int i = e * 32 + tid / 8, cc = c0 + tid % 8 * 4, to = image_at(i, tid % 8 * 4, 2);
                float a[4], u[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = i < live && cc + j < p.dv;
                    a[j] = in ? na[e][j] : 0.f, u[j] = in ? nu[e][j] : 0.f, y[j] = in ? (float)ny[e][j] : 0.f;
                    db[e] = fmaf(a[j], u[j], db[e]);
                }
                put_terms<3>(ix, to, SB, a);
                put_terms<3>(iw, to, SB, u);
                put_terms<N>(iy, to, SB, y);
            }
            __syncthreads();
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                if (wave < KT) {
                    const auto fetch = [&](const float *from, float (&v8)[8]) {
                        float lo[4], hi[4];
                        const float *row = from + (int64_t)min(d, p.dk - 1) * p.dv;
                        load4<VEC>(lo, row, c0 + st * 16 + 4 * half, p.dv, d < p.dk);
                        load4<VEC>(hi, row, c0 + st * 16 + 4 * half + 8, p.dv, d < p.dk);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v8[j] = lo[j], v8[4 + j] = hi[j];
                    };
                    float s8[8], d8[8];
                    fetch(S, s8), fetch(D, d8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) inner = fmaf(s8[j], d8[j], inner);
                    const Frag<3> fs = split<3>(s8), fd = split<3>(d8);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        multiply<2>(ys[i], piece<N>(iy, i * 2 + st, SB), fs);
                        multiply<2>(xs[i], piece<3>(ix, i * 2 + st, SB), fs);
                        multiply<2>(wd[i], piece<3>(iw, i * 2 + st, SB), fd);
                    }
                }
                if (wave < MT * MT) {
                    const Frag<3> fw = piece<3>(iw, wave % MT * 2 + st, SB);
                    multiply<2>(xw, piece<3>(ix, wave / MT * 2 + st, SB), fw);
                    multiply<2>(yw, piece<N>(iy, wave / MT * 2 + st, SB), fw);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < MT; ++e) {
#pragma unroll
            for (int o = 1; o < 8; o *= 2) db[e] += __shfl_xor(db[e], o, 64);
            if (tid % 8 == 0) dotb[e * 32 + tid / 8] = db[e];
        }
        __syncthreads();                                 // the slabs have been read
        if (wave < MT * MT) {
            const int bi = wave / MT, bj = wave % MT, j = bj * 32 + col;
            f32x16 kk = zeros16(), qk = zeros16();
            if (bi >= bj) {
                if ((p.dk & 3) == 0) products(kk, qk, bi, bj, std::true_type());
                else products(kk, qk, bi, bj, std::false_type());
            }
            float before = 0.f;                          // of this block: rows from j on, columns before j
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = bi * 32 + acc_row(r);
                const float e = i >= j ? exp2f((float)(G[i] - G[j])) * beta[j] : 0.f;
                const float hij = i > j ? -beta[i] * e * xw[r] : 0.f, jij = p.scale * e * yw[r];
                Hm[i * LD + j] = hij;
                Jm[i * LD + j] = jij;
                if (bi < bj) continue;
                const float to = half_sums(fmaf(hij * rk[i], kk[r], jij * rq[i] * qk[r]) * rk[j]);
                const float under = __shfl_up(to, 1, 32);
                before += col > 0 && i >= j ? under : 0.f;
                if (bi > bj && col == 31) pairs[1][i] = to;      // a whole row of the block below
            }
            before = both_halves(before);
            if (bi >= bj && half == 0) pairs[bi - bj][j] = before;
        }
        // the states' shares, with their rows' factors, where the pairs' are added
        if (wave < KT) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    float kv[4], qv[4];
                    four(ikt, i * 32 + acc_row(r4 * 4), kv);
                    four(iqt, i * 32 + acc_row(r4 * 4), qv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = r4 * 4 + j, row = i * 32 + acc_row(r);
                        const float rise = exp2f((float)G[row]), fall = exp2f((float)(G[C - 1] - G[row])) * beta[row];
                        ys[i][r] *= p.scale * rise;
                        xs[i][r] *= -rise * beta[row];
                        wd[i][r] *= fall;
                        const float own = half_sums(fmaf(rq[row] * qv[j], ys[i][r], rk[row] * kv[j] * xs[i][r]));
                        const float end = half_sums(rk[row] * kv[j] * wd[i][r]);
                        if (col == 31) dots[wave][row] = own, dote[wave][row] = end;
                        xs[i][r] += wd[i][r];
                    }
                }
        }
        __syncthreads();
        if (wave < KT) {
#pragma unroll
            for (int cs = 0; cs < CS; ++cs) {
                const Frag<N> fk = piece<N>(ikt, wave * CS + cs, KB), fq = piece<N>(iqt, wave * CS + cs, KB);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float a[8], e[8], u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = i * 32 + col, t = cs * 16 + 8 * (j >> 2) + 4 * half + (j & 3);
                        a[j] = Jm[r * LD + t] * rk[t];
                        e[j] = Jm[t * LD + r] * rq[t];
                        u[j] = (r > t ? Hm[r * LD + t] : Hm[t * LD + r]) * rk[t];
                    }
                    multiply<2>(ys[i], split<3>(a), fk);
                    multiply<2>(xs[i], split<3>(e), fq);
                    multiply<2>(xs[i], split<3>(u), fk);
                    in_order();
                }
            }
            if (SHARED) {
#pragma unroll
                for (int i = 0; i < MT; ++i) allq[i] += ys[i], allk[i] += xs[i];
            }
        }
        inner = lanes_sum(inner);
        if (lane == 0) total[wave] = inner;
        __syncthreads();
        if (wave == 0) {
            // lane t's decay: own, and of the blocks on the diagonal what is before it; the block
            // below them adds its columns before t, or its rows from t on
            float all = 0.f, own = 0.f, ends = 0.f, g = 0.f, under = 0.f;
#pragma unroll
            for (int i = 0; i < KT; ++i) all += total[i];
            if (lane < C) {
#pragma unroll
                for (int i = 0; i < KT; ++i) own += dots[i][lane], ends += dote[i][lane];
                g = pairs[0][lane];
                if (MT == 2) under = pairs[1][lane];
            }
#pragma unroll
            for (int o = 1; o < C; o *= 2) {
                const float z = __shfl_down(own, o, 64), u = __shfl_up(ends, o, 64);
                if (lane + o < C) own += z;
                if (lane >= o) ends += u;
            }
            if (MT == 2) {
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const float u = __shfl_down(under, o, 32);
                    if (half == 1 && col + o < 32) under += u;
                }
            }
            const float z = __shfl_up(ends, 1, 64);
            g = (g + under) + (own + (lane > 0 ? z : 0.f)) + exp2f((float)G[C - 1]) * all;
            if (lane < rows) {
                const int64_t row = row0 + (int64_t)lane * p.B;
                p.dg[row * p.lddg + h] = lane < live ? g : 0.f;
                p.dbeta[row * p.lddb + h] = lane < live ? dotb[lane] : 0.f;
            }
        }
    }
    // over the lengths: d = r (d^ - x^ (x^ . d^)), x^ = r x
    if (p.unit) {
        __syncthreads();
        if (wave < KT)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    float qv[4], kv[4];
                    four(iqt, i * 32 + acc_row(r4 * 4), qv);
                    four(ikt, i * 32 + acc_row(r4 * 4), kv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = r4 * 4 + j, row = i * 32 + acc_row(r);
                        const float dotq = half_sums(rq[row] * qv[j] * allq[i][r]);
                        const float dotk = half_sums(rk[row] * kv[j] * allk[i][r]);
                        if (col == 31) dots[wave][row] = dotq, dote[wave][row] = dotk;
                    }
                }
        __syncthreads();
    }
    if (wave >= KT || d >= p.dk) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            float qv[4], kv[4];
            four(iqt, i * 32 + acc_row(r4 * 4), qv);
            four(ikt, i * 32 + acc_row(r4 * 4), kv);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r4 * 4 + j, row = i * 32 + acc_row(r);
                if (row >= rows) continue;
                float gq = allq[i][r], gk = allk[i][r];
                if (p.unit) {
                    float dotq = 0.f, dotk = 0.f;
#pragma unroll
                    for (int t = 0; t < KT; ++t) dotq += dots[t][row], dotk += dote[t][row];
                    gq = rq[row] * fmaf(-rq[row] * qv[j], dotq, gq);
                    gk = rk[row] * fmaf(-rk[row] * kv[j], dotk, gk);
                }
                const int64_t to = row0 + (int64_t)row * p.B;
                dq[to * p.lddq + d] = (T)(row < live ? gq : 0.f);
                dk[to * p.lddk + d] = (T)(row < live ? gk : 0.f);
            }
        }
}

template <typename T, int KT>
void backward(const DeltaArgs &a, hipStream_t st) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms, KB = C * KT * 64, MB = tri_pieces<C>() * kPiece;
    const int heads = a.B * a.H;
    const ChainGrid g = chain_grid((a.dv + 15) / 16, C, KT);
    const int chain = N * KB * 2 + 6 * MB + factor_bytes<C>();
    const dim3 all((unsigned)(a.chunks * heads));
    if (a.dk % 4 == 0) hipLaunchKernelGGL((k_delta_prep<T, KT, true, true>), all, dim3(64), 0, st, a);
    else hipLaunchKernelGGL((k_delta_prep<T, KT, true, false>), all, dim3(64), 0, st, a);
    if (a.segments > 1) {
        hipLaunchKernelGGL((k_delta_back_chain<T, KT, false>), dim3((unsigned)((a.segments - 1) * heads), g.groups), dim3(g.threads),
                           chain, st, a);
        delta_join(a, a.dfinal, true, st);
    }
    hipLaunchKernelGGL((k_delta_back_chain<T, KT, true>), dim3((unsigned)(a.segments * heads), g.groups), dim3(g.threads), chain, st,
                       a);
    const dim3 own((unsigned)(a.chunks * a.B * a.HK));
    const int lds = std::max((6 + N) * C / 32 * 2 * kPiece, 2 * C * (C + 4) * 4) + 2 * N * KB;
    // SHARED where heads share a key head: its sums cost a CU its second workgroup (without them
    // 8192 x 4 x 6 heads 128 x 130 bf16 1816 -> 1558 us backwards, 4096 x 2 x 6 heads 96 x 97 fp32 548 -> 439)
    const auto run = [&](auto vec, auto shared) {
        hipLaunchKernelGGL((k_delta_grads<T, KT, decltype(vec)::value, decltype(shared)::value>), own, dim3(256), lds, st, a);
    };
    const std::true_type yes;
    const std::false_type no;
    const bool vec = a.dv % 4 == 0, shared = a.H > a.HK;
    if (vec) shared ? run(yes, yes) : run(yes, no);
    else shared ? run(no, yes) : run(no, no);
}

template <typename T>
void backward(const DeltaArgs &a, hipStream_t st) {
    switch ((a.dk + 31) / 32) {
        case 1: return backward<T, 1>(a, st);
        case 2: return backward<T, 2>(a, st);
        case 3: return backward<T, 3>(a, st);
        default: return backward<T, 4>(a, st);
    }
}

// No positions: the gradient passes through.
__global__ void __launch_bounds__(256) k_delta_pass(const float *from, float *to, int64_t n) {
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += gridDim.x * (int64_t)256) to[i] = from ? from[i] : 0.f;
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" fi_status fi_delta_backward(const fi_delta_desc *desc, const void *q, const void *k, const void *v,
                                       const float *decay, const float *beta, const float *state, const int32_t *lengths,
                                       const void *saved, const void *dy, const float *dfinal, void *dq, void *dk, void *dv,
                                       float *ddecay, float *dbeta, float *dstate, void *workspace, void *stream) {
    static const char *call = "fi_delta_backward";
    if (const char *why = delta_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (desc->T > 0 && (!q || !k || !v || !decay || !beta || !saved || !dy || !dq || !dk || !dv || !ddecay || !dbeta || !workspace))
        return op_fail(FI_EINVAL, call, "q, k, v, decay, beta, saved, dy, their gradients and the workspace are required");
    const size_t es = value_bytes(desc->dtype);
    if (!aligned(es, {q, k, v, dy, dq, dk, dv}) || !aligned(4, {decay, beta, state, lengths, dfinal, ddecay, dbeta, dstate}) ||
        !aligned(256, {saved, workspace}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const DeltaPlan d = delta_plan(desc);
    DeltaArgs a = {};
    delta_args(desc, d, a);
    const int64_t rows = a.T * a.B;
    const size_t qk = (size_t)a.HK * a.dk * es, vb = (size_t)a.H * a.dv * es, hb = (size_t)a.H * 4;
    const size_t sb = (size_t)a.B * a.H * a.dk * a.dv * 4, lb = (size_t)a.B * 4;
    const size_t sv = fi_delta_saved_bytes(desc), ws = fi_delta_workspace_bytes(desc, 1);
    const View out[] = {{dq, rows, qk, (size_t)a.lddq * es}, {dk, rows, qk, (size_t)a.lddk * es}, {dv, rows, vb, (size_t)a.lddv * es},
                        {ddecay, rows, hb, (size_t)a.lddg * 4}, {dbeta, rows, hb, (size_t)a.lddb * 4}, {dstate, 1, sb, sb},
                        {workspace, 1, ws, ws}};
    const View in[] = {{q, rows, qk, (size_t)a.ldq * es}, {k, rows, qk, (size_t)a.ldk * es}, {v, rows, vb, (size_t)a.ldv * es},
                       {decay, rows, hb, (size_t)a.ldg * 4}, {beta, rows, hb, (size_t)a.ldb * 4}, {state, 1, sb, sb},
                       {lengths, 1, lb, lb}, {saved, 1, sv, sv}, {dy, rows, vb, (size_t)a.lddy * es}, {dfinal, 1, sb, sb}};
    if (outputs_meet(out, 7, in, 10)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    const hipStream_t st = (hipStream_t)stream;
    if (a.T == 0) {
        if (dstate)
            hipLaunchKernelGGL(k_delta_pass, dim3((unsigned)std::min<size_t>((sb / 4 + 255) / 256, 4096)), dim3(256), 0, st, dfinal,
                               dstate, (int64_t)(sb / 4));
        return op_launched(call);
    }
    a.q = q, a.k = k, a.v = v, a.g = decay, a.beta = beta, a.lengths = lengths, a.dy = dy, a.dfinal = dfinal;
    a.dq = dq, a.dk_out = dk, a.dv_out = dv, a.dg = ddecay, a.dbeta = dbeta, a.dstate = dstate;
    char *w = (char *)workspace;
    a.images = w, w += d.images;
    a.factors = (float *)w, w += d.factors;
    a.ends = (float *)w, w += d.ends;
    a.x = (float *)w, w += d.rows;
    a.starts = (float *)w, w += d.local;
    a.local = (float *)w;
    char *s = (char *)saved;
    a.states = (float *)s, s += d.states;
    a.w = (float *)s, s += d.rows;
    a.maps = (float *)s;
    if (desc->dtype == FI_F32) backward<float>(a, st);
    else if (desc->dtype == FI_BF16) backward<bf16_t>(a, st);
    else backward<f16_t>(a, st);
    return op_launched(call);
}
