// The gated delta rule (fi_delta_*): the forward pass in chunks, and position by
// position where there are few.
#include "fi_delta.h"

namespace fi {

namespace {

enum { CHAIN_LOCAL, CHAIN_FULL };

// LDS of the whole sequence's kernel, and whether P's last term comes into k's place there
// after k's last use: with a place of its own it would leave a CU one workgroup where
// without it there are two (bf16 keys of over 96 channels).
constexpr int kTwoWorkgroups = 80 * 1024;
template <typename T, int KT>
constexpr int full_bytes() {
    constexpr int C = DeltaType<T>::chunk;
    return 3 * DeltaType<T>::terms * C * KT * 64 + 6 * tri_pieces<C>() * kPiece + factor_bytes<C>();
}
template <typename T, int KT>
constexpr bool p_late() {
    return full_bytes<T, KT>() > kTwoWorkgroups &&
           full_bytes<T, KT>() - tri_pieces<DeltaType<T>::chunk>() * kPiece <= kTwoWorkgroups;
}

// The sequence of a segment's chunks, 16 columns a wave (blockIdx.y: a workgroup's).
// FULL: from the state before the segment; y, the states before each chunk and w where
// they are kept, the last state.  LOCAL: from nothing, only the state at the end; the
// columns behind the state's are those of the map (v = 0, from a unit column).
// What a chunk needs is on its way while the one before it runs: k and q in registers,
// M, P and the factors past them into LDS as soon as nobody reads the last ones.
// 131072 positions of 9 heads of 96 bf16: FULL 612 us (56 segments of 37 chunks, two
// workgroups a CU, 16 us a chunk), LOCAL 756.  Of a chunk's 36000 cycles a wave issues
// 180 products (2900) and 790 others (3200); the loads account for 100 us, bringing k
// and q into LDS for 80; the rest waits in the phases' chain of products, terms and four
// barriers.  Wider waves (32 columns) ran no faster, nor did all of a step's operands
// read ahead of it or v and y by whole vectors (653 and 585 us where it took 550).
template <typename T, int KT, int MODE>
__global__ void __launch_bounds__(512, 4) k_delta_chain(DeltaArgs p) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms;
    constexpr int MT = C / 16, CS = C / 32, DT = KT * 2, DK = KT * 32;
    constexpr int KB = C * DK * 2, MB = tri_pieces<C>() * kPiece;    // bytes of a term
    constexpr bool FULL = MODE == CHAIN_FULL, LATE = FULL && p_late<T, KT>();
    extern __shared__ __align__(16) char lds[];
    char *const ik = lds, *const ikt = ik + N * KB, *const im = ikt + N * KB;
    char *const ip = im + 3 * MB, *const iq = ip + (LATE ? 2 : 3) * MB;   // FULL only
    char *const ip2 = LATE ? ik : ip + 2 * MB;                 // P's last term
    char *const ff = FULL ? iq + N * KB : ip;
    const float *const f = reinterpret_cast<const float *>(ff);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.B * p.H, seg = blockIdx.x / heads, bh = blockIdx.x % heads, b = bh / p.H, h = bh % p.H;
    const int tiles = (p.dv + 15) / 16, tile = blockIdx.y * (int)(blockDim.x >> 6) + wave;
    const bool map = !FULL && tile >= tiles, idle = map ? (tile - tiles) * 16 >= p.dk : tile >= tiles;
    const int column = (map ? tile - tiles : tile) * 16 + (lane & 15), width = map ? p.dk : p.dv;
    const bool mine = column < width && !idle;
    const int64_t length = delta_length(p, b);
    const int hk = h / (p.H / p.HK);
    const int64_t size = (int64_t)p.dk * p.dv;

    f32x4 S[DT];
    const float *from = !FULL ? nullptr : p.segments > 1 ? p.starts + ((int64_t)seg * heads + bh) * size
                                        : p.state        ? p.state + bh * size
                                                         : nullptr;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = map && t * 16 + tile_row(r) == column ? 1.f : 0.f;
    if (from) load_state(S, from, p.dk, p.dv, column);
    const auto keep = [&](float *to, int w) { store_state(to, S, p.dk, w, idle ? w : column); };

    const T *const q = static_cast<const T *>(p.q) + hk * p.dk, *const k = static_cast<const T *>(p.k) + hk * p.dk;
    const T *const v = static_cast<const T *>(p.v) + (int64_t)h * p.dv;
    const int64_t first = seg * p.per, last = min(p.chunks, first + p.per);
    const int64_t stop = min(last, (length + C - 1) / C);      // chunks behind it hold nothing
    Stage<T, C, DK, true> sk, sq;
    T vs[MT][4];
    const auto ahead = [&](int64_t c) {
        const int64_t t0 = c * C;
        const int live = (int)min<int64_t>(C, length - t0);
        sk.load(k + (t0 * p.B + b) * p.ldk, (unsigned)(p.B * p.ldk), p.dk, live);
        if (FULL) sq.load(q + (t0 * p.B + b) * p.ldq, (unsigned)(p.B * p.ldq), p.dk, live);
    };
    const auto matrices = [&](int64_t c) {                     // M, P and the factors; v
        const int64_t at = c * heads + bh;
        bring(im, p.images + at * image_bytes<T>(), (LATE ? 5 : FULL ? 6 : 3) * MB);
        bring(ff, (const char *)(p.factors + at * kDeltaFactors * C), factor_bytes<C>());
        if (!map)
            load_column<T, MT>(vs, v + (c * C * p.B + b) * p.ldv, min(column, p.dv - 1), (unsigned)(p.B * p.ldv),
                               (int)min<int64_t>(C, length - c * C));
    };
    if (first < stop) ahead(first), matrices(first);
    for (int64_t c = first; c < stop; ++c) {
        const int64_t t0 = c * C, at = c * heads + bh;
        const int rows = (int)min<int64_t>(C, p.T - t0), live = (int)min<int64_t>(C, length - t0);
        __syncthreads();
        sk.put(p.dk, live, ik, ikt);
        if (FULL) sq.put(p.dk, live, iq, nullptr);
        __syncthreads();
        if (FULL && p.states) keep(p.states + at * size, p.dv);

        f32x4 R[MT], Y[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) R[i] = Y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KT; ++ks) {
            const Frag<3> s = step_of<3>(S, ks);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                multiply<2>(R[i], piece<N>(ik, i * KT + ks, KB), s);
                if (FULL) multiply<2>(Y[i], piece<N>(iq, i * KT + ks, KB), s);
            }
            in_order();
        }
        arrived();
        __syncthreads();
        if (LATE) bring(ip2, p.images + at * image_bytes<T>() + 5 * MB, MB);   // k has been read
        // v - e^G K S, and w = M of it
        const int vlive = anew(map ? 0 : live);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + tile_row(r);
                R[i][r] = fmaf(-f[row], R[i][r], row < vlive ? (float)vs[i][r] : 0.f);
            }
        f32x4 W[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) W[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            const Frag<3> s = step_of<3>(R, cs);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                if (tri_in<C, false>(i, cs)) multiply<2>(W[i], piece<3>(im, tri_at<C, false>(i, cs), MB), s);
            in_order();
        }
        if (LATE) {
            arrived();
            __syncthreads();
        }
        if (!FULL && c + 1 < stop) ahead(c + 1);
        if (FULL) {
            if (p.w && mine) store_column<float, MT>(p.w + at * C * p.dv, column, p.dv, W, C, C);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) Y[i][r] *= f[C + i * 16 + tile_row(r)];
#pragma unroll
            for (int cs = 0; cs < CS; ++cs) {
                const Frag<3> s = step_of<3>(W, cs);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    if (tri_in<C, false>(i, cs)) {
                        const Frag<2> p01 = piece<2>(ip, tri_at<C, false>(i, cs), MB);
                        multiply<2>(Y[i], Frag<3>{p01.t[0], p01.t[1], piece<1>(ip2, tri_at<C, false>(i, cs), MB).t[0]}, s);
                    }
                in_order();
            }
            if (mine)
                store_column<T, MT>(static_cast<T *>(p.y) + (int64_t)h * p.dv + (t0 * p.B + b) * p.ldy, column,
                                    (unsigned)(p.B * p.ldy), Y, rows, live);
        }
        // the whole sequence's next k and q begin behind y: ahead of it they would push v's
        // loads into scratch memory (131072 positions of 9 heads of 96 1840 us in place of 1650)
        if (FULL && c + 1 < stop) ahead(c + 1);
        const float decay = f[4 * C];
#pragma unroll
        for (int t = 0; t < DT; ++t) S[t] *= decay;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) W[i][r] *= f[2 * C + i * 16 + tile_row(r)];
        __syncthreads();
        if (c + 1 < stop) matrices(c + 1);
#pragma unroll
        for (int cs = 0; cs < CS; ++cs) {
            const Frag<3> s = step_of<3>(W, cs);
#pragma unroll
            for (int t = 0; t < DT; ++t) multiply<2>(S[t], piece<N>(ikt, t * CS + cs, KB), s);
            in_order();
        }
    }
    if (!FULL) {
        // the map as it is for the backward pass, transposed for joining forwards: either
        // way a wave then reads it along its lanes
        if (map) {
            const int64_t to = ((int64_t)seg * heads + bh) * p.dk * p.dk;
            if (p.states) keep(p.maps + to, p.dk);
            if (!idle && column < p.dk)
#pragma unroll
                for (int t = 0; t < DT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (t * 16 + tile_row(r) < p.dk) p.mapst[to + column * p.dk + t * 16 + tile_row(r)] = S[t][r];
        } else keep(p.local + ((int64_t)seg * heads + bh) * size, p.dv);
        return;
    }
    // behind the sequence's end: y = 0, the state as it is
    for (int64_t c = max(first, stop); c < last; ++c) {
        const int64_t t0 = c * C;
        const int rows = (int)min<int64_t>(C, p.T - t0);
        T *const y = static_cast<T *>(p.y) + (int64_t)h * p.dv + (t0 * p.B + b) * p.ldy + column;
        if (mine)
            for (int i = lane >> 4; i < rows; i += 4) y[i * p.B * p.ldy] = (T)0.f;
    }
    if (seg == p.segments - 1 && p.final) keep(p.final + bh * size, p.dv);
}

// starts[s + 1] = maps[s] starts[s] + local[s] (backwards starts[s - 1] = maps[s]^T
// starts[s] + local[s]): a workgroup 32 columns of a head, a wave 32 rows, whose share
// of the next map is on its way meanwhile; the state passes through LDS as an image.
template <int KT, bool BACK>
__global__ void __launch_bounds__(KT * 64) k_delta_join(DeltaArgs p, const float *first) {
    constexpr int KS = KT * 2;
    __shared__ __align__(16) char image[2][3 * KS * kPiece];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const int heads = p.B * p.H, bh = blockIdx.x, column = blockIdx.y * 32 + (lane & 31), at = min(column, p.dv - 1);
    const int64_t size = (int64_t)p.dk * p.dv, msize = (int64_t)p.dk * p.dk;
    const int row = min(wave * 32 + (lane & 31), p.dk - 1);
    const bool in = wave * 32 + (lane & 31) < p.dk;
    f32x16 S;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int d = wave * 32 + acc_row(r);
        const float s = first ? first[bh * size + (int64_t)min(d, p.dk - 1) * p.dv + at] : 0.f;
        S[r] = d < p.dk ? s : 0.f;
    }
    float map[KS][8], local[16];
    const auto ahead = [&](int s) {
        const float *m = (BACK ? p.maps : p.mapst) + ((int64_t)s * heads + bh) * msize, *l = p.local + ((int64_t)s * heads + bh) * size + at;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = min(ks * 16 + 8 * (j >> 2) + 4 * half + (j & 3), p.dk - 1);
                map[ks][j] = m[k * p.dk + row];
            }
#pragma unroll
        for (int r = 0; r < 16; ++r) local[r] = l[min(wave * 32 + acc_row(r), p.dk - 1) * p.dv];
    };
    const int s0 = BACK ? p.segments - 1 : 0, step = BACK ? -1 : 1;
    ahead(s0);
    for (int n = 0; n < p.segments; ++n) {
        const int s = s0 + n * step;
        float *to = p.starts + ((int64_t)s * heads + bh) * size;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int d = wave * 32 + acc_row(r);
            if (d < p.dk && column < p.dv) to[d * p.dv + column] = S[r];
        }
        if (n + 1 == p.segments) break;
        char *const im = image[n & 1];
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const float x[4] = {S[r], S[r + 1], S[r + 2], S[r + 3]};
            put_terms<3>(im, image_at(lane & 31, wave * 32 + acc_row(r), KS), KS * kPiece, x);
        }
        f32x16 part[2] = {zeros16(), zeros16()};
        Frag<3> fm[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = in && ks * 16 + 8 * (j >> 2) + 4 * half + (j & 3) < p.dk ? map[ks][j] : 0.f;
            fm[ks] = split<3>(x);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) part[0][r] = wave * 32 + acc_row(r) < p.dk ? local[r] : 0.f;
        if (n + 2 < p.segments) ahead(s + step);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) multiply<2>(part[ks & 1], fm[ks], piece<3>(im, ks, KS * kPiece));
#pragma unroll
        for (int r = 0; r < 16; ++r) S[r] = part[0][r] + part[1][r];
    }
}

// Position by position, for a few of them: a workgroup 32 columns of a head, a thread
// four columns of every 32nd row, held in registers (one position of 8 x 9 heads of 96
// 7.1 us, of which the state's 5.3 MB are one: two loads that wait for each other, two
// sums over the workgroup and the launch).  Both sums over the rows, k . S
// and q . S, are taken of the state before the position:
// y = scale (a q.S + (k.q) u), u = b (v - a k.S).
template <typename T>
__global__ void __launch_bounds__(256) k_delta_steps(DeltaArgs p) {
    constexpr int ROWS = kDeltaMaxK / 32;
    __shared__ float ks[kDeltaMaxK], qs[kDeltaMaxK];
    __shared__ float4 join[2][4][8];
    __shared__ float dots[3][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cg = tid & 7, rg = tid >> 3;
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.HK), column = blockIdx.y * 32 + cg * 4;
    const int64_t length = delta_length(p, b);
    const bool vec = (p.dv & 3) == 0;
    float S[ROWS][4];
    const float *from = p.state ? p.state + (int64_t)bh * p.dk * p.dv : nullptr;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = rg + i * 32;
        if (from && vec) load4<true>(S[i], from + (int64_t)min(row, p.dk - 1) * p.dv, column, p.dv, row < p.dk);
        else if (from) load4<false>(S[i], from + (int64_t)min(row, p.dk - 1) * p.dv, column, p.dv, row < p.dk);
        else S[i][0] = S[i][1] = S[i][2] = S[i][3] = 0.f;
    }
    for (int64_t t = 0; t < p.T; ++t) {
        const int64_t row = t * p.B + b;
        T *const y = static_cast<T *>(p.y) + row * p.ldy + (int64_t)h * p.dv;
        if (t >= length) {
            if (rg == 0)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (column + j < p.dv) y[column + j] = (T)0.f;
            continue;
        }
        __syncthreads();
        float kk = 0.f, qq = 0.f, kq = 0.f;
        if (tid < kDeltaMaxK) {
            const bool in = tid < p.dk;
            const float a = in ? (float)static_cast<const T *>(p.k)[row * p.ldk + hk * p.dk + tid] : 0.f;
            const float c = in ? (float)static_cast<const T *>(p.q)[row * p.ldq + hk * p.dk + tid] : 0.f;
            ks[tid] = a, qs[tid] = c;
            kk = a * a, qq = c * c, kq = a * c;
        }
        kk = lanes_sum(kk), qq = lanes_sum(qq), kq = lanes_sum(kq);
        if (lane == 0) dots[0][wave] = kk, dots[1][wave] = qq, dots[2][wave] = kq;
        __syncthreads();
        const float rk = p.unit ? 1.f / sqrtf(dots[0][0] + dots[0][1] + kDeltaUnit) : 1.f;
        const float rq = p.scale * (p.unit ? 1.f / sqrtf(dots[1][0] + dots[1][1] + kDeltaUnit) : 1.f);
        float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float a = ks[rg + i * 32], c = qs[rg + i * 32];
#pragma unroll
            for (int j = 0; j < 4; ++j) pk[j] = fmaf(a, S[i][j], pk[j]), pq[j] = fmaf(c, S[i][j], pq[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 8; s < 64; s *= 2) pk[j] += __shfl_xor(pk[j], s, 64), pq[j] += __shfl_xor(pq[j], s, 64);
        if (lane < 8) {
            join[0][wave][cg] = make_float4(pk[0], pk[1], pk[2], pk[3]);
            join[1][wave][cg] = make_float4(pq[0], pq[1], pq[2], pq[3]);
        }
        __syncthreads();
        float v[4];
        load4<false>(v, static_cast<const T *>(p.v) + row * p.ldv + (int64_t)h * p.dv, column, p.dv, true);
        const float g = p.g[row * p.ldg + h], beta = p.beta[row * p.ldb + h], a = exp2f(g * kLog2e);
        const float cross = (dots[2][0] + dots[2][1]) * rk * rq;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) sk += (&join[0][w][cg].x)[j], sq += (&join[1][w][cg].x)[j];
            const float u = beta * fmaf(-a * rk, sk, v[j]);
            if (rg == 0 && column + j < p.dv) y[column + j] = (T)fmaf(a * rq, sq, cross * u);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) S[i][j] = fmaf(ks[rg + i * 32] * rk, u, a * S[i][j]);
        }
    }
    if (!p.final) return;
    float *const to = p.final + (int64_t)bh * p.dk * p.dv;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = rg + i * 32;
        if (row < p.dk)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (column + j < p.dv) to[(int64_t)row * p.dv + column + j] = S[i][j];
    }
}

// Up to as many positions run one by one: 1.8 us each, where the chunk's two launches take
// 31 to 40 us at any number up to 64 (8, 14, 24 positions one by one and in a chunk: 9
// heads of 96 19 and 32, 30 and 32, 48 and 32 us, 8 x 9 the same, 64 heads of 128 20 and
// 40, 31 and 40, 49 and 40).  Very many or very narrow heads turn earlier: 32 x 16 heads of
// 128 55 and 59, 83 and 60, 2 heads of 32 18 and 23, 29 and 23.
constexpr int64_t kDeltaSteps = 14;

template <typename T, int KT>
void forward(const DeltaArgs &a, const DeltaPlan &d, hipStream_t st) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms;
    constexpr int KB = C * KT * 64, MB = tri_pieces<C>() * kPiece, FB = factor_bytes<C>();
    const int heads = a.B * a.H;
    const dim3 all((unsigned)(a.chunks * heads));
    if (a.dk % 4 == 0) hipLaunchKernelGGL((k_delta_prep<T, KT, false, true>), all, dim3(64), 0, st, a);
    else hipLaunchKernelGGL((k_delta_prep<T, KT, false, false>), all, dim3(64), 0, st, a);
    if (a.segments > 1) {
        // the last segment's map is the backward pass's alone
        const int parts = a.states ? a.segments : a.segments - 1;
        const ChainGrid g = chain_grid((a.dv + 15) / 16 + (a.dk + 15) / 16, C, KT);
        hipLaunchKernelGGL((k_delta_chain<T, KT, CHAIN_LOCAL>), dim3((unsigned)(parts * heads), g.groups), dim3(g.threads),
                           N * KB * 2 + 3 * MB + FB, st, a);
        delta_join(a, a.state, false, st);
    }
    const ChainGrid g = chain_grid((a.dv + 15) / 16, C, KT);
    constexpr int full = full_bytes<T, KT>() - (p_late<T, KT>() ? MB : 0);
    hipLaunchKernelGGL((k_delta_chain<T, KT, CHAIN_FULL>), dim3((unsigned)(a.segments * heads), g.groups), dim3(g.threads),
                       full, st, a);
}

template <typename T>
void forward(const DeltaArgs &a, const DeltaPlan &d, bool steps, hipStream_t st) {
    if (steps)
        hipLaunchKernelGGL((k_delta_steps<T>), dim3(a.B * a.H, (a.dv + 31) / 32), dim3(256), 0, st, a);
    else if (d.KT == 1) forward<T, 1>(a, d, st);
    else if (d.KT == 2) forward<T, 2>(a, d, st);
    else if (d.KT == 3) forward<T, 3>(a, d, st);
    else forward<T, 4>(a, d, st);
}

}  // namespace

const char *delta_check(const fi_delta_desc *q) {
    if (!q) return "null descriptor";
    if (q->T < 0 || q->T > (int64_t(1) << 23)) return "T is not in 0 .. 2^23";
    if (q->batch < 1 || q->key_heads < 1 || q->heads < 1) return "batch >= 1, key_heads >= 1 and heads >= 1 are required";
    if (q->heads % q->key_heads) return "heads is no multiple of key_heads";
    if (q->dk < 1 || q->dk > kDeltaMaxK) return "dk is not in 1 .. 128";
    if (q->dv < 1 || q->dv > kDeltaMaxV) return "dv is not in 1 .. 1024";
    if (!value_type(q->dtype)) return "dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->unit != 0 && q->unit != 1) return "unit is not 0 or 1";
    if (!(q->scale == q->scale)) return "scale is not a number";
    if ((int64_t)q->batch * q->heads > int64_t(1) << 20) return "batch * heads is over 2^20";
    const int C = delta_chunk(q->dtype);
    // a launch has less than 2^32 threads, 256 of them a chunk and key head backwards
    if ((q->T + C - 1) / C * q->batch * q->heads >= int64_t(1) << 24) return "too large: chunks * batch * heads is not below 2^24";
    const int64_t qk = (int64_t)q->key_heads * q->dk, v = (int64_t)q->heads * q->dv, h = q->heads;
    const int64_t ld[][2] = {{q->ld_q, qk}, {q->ld_k, qk}, {q->ld_v, v}, {q->ld_decay, h}, {q->ld_beta, h}, {q->ld_y, v},
                             {q->ld_dy, v}, {q->ld_dq, qk}, {q->ld_dk, qk}, {q->ld_dv, v}, {q->ld_ddecay, h},
                             {q->ld_dbeta, h}};
    for (auto &l : ld) {
        if (l[0] != 0 && l[0] < l[1]) return "a row pitch is less than its row";
        if (l[0] > (int64_t(1) << 24) / q->batch || l[1] > (int64_t(1) << 24) / q->batch)
            return "the rows of a position are over 2^24 elements";
    }
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    return nullptr;
}

void delta_args(const fi_delta_desc *q, const DeltaPlan &d, DeltaArgs &a) {
    a.T = q->T, a.chunks = d.chunks, a.per = d.per, a.segments = d.segments;
    a.B = q->batch, a.HK = q->key_heads, a.H = q->heads, a.dk = q->dk, a.dv = q->dv, a.unit = q->unit, a.scale = q->scale;
    const int64_t qk = (int64_t)a.HK * a.dk, v = (int64_t)a.H * a.dv;
    a.ldq = pitch_or(q->ld_q, qk), a.ldk = pitch_or(q->ld_k, qk), a.ldv = pitch_or(q->ld_v, v);
    a.ldg = pitch_or(q->ld_decay, a.H), a.ldb = pitch_or(q->ld_beta, a.H), a.ldy = pitch_or(q->ld_y, v);
    a.lddy = pitch_or(q->ld_dy, v), a.lddq = pitch_or(q->ld_dq, qk), a.lddk = pitch_or(q->ld_dk, qk);
    a.lddv = pitch_or(q->ld_dv, v), a.lddg = pitch_or(q->ld_ddecay, a.H), a.lddb = pitch_or(q->ld_dbeta, a.H);
}

template <int KT>
static void join(const DeltaArgs &a, const float *first, bool back, hipStream_t st) {
    const dim3 grid(a.B * a.H, (a.dv + 31) / 32), block(KT * 64);
    if (back) hipLaunchKernelGGL((k_delta_join<KT, true>), grid, block, 0, st, a, first);
    else hipLaunchKernelGGL((k_delta_join<KT, false>), grid, block, 0, st, a, first);
}

void delta_join(const DeltaArgs &a, const float *first, bool back, hipStream_t st) {
    switch ((a.dk + 31) / 32) {
        case 1: return join<1>(a, first, back, st);
        case 2: return join<2>(a, first, back, st);
        case 3: return join<3>(a, first, back, st);
        default: return join<4>(a, first, back, st);
    }
}

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_delta_saved_bytes(const fi_delta_desc *desc) {
    if (delta_check(desc)) return 0;
    const DeltaPlan d = delta_plan(desc);
    return d.states + d.rows + d.maps + 256;
}

size_t fi_delta_workspace_bytes(const fi_delta_desc *desc, int backward) {
    if (delta_check(desc)) return 0;
    if (backward) {
        const DeltaPlan d = delta_plan(desc);
        return d.images + d.factors + d.ends + d.rows + 2 * d.local + 256;
    }
    const DeltaPlan d = delta_plan(desc);
    return d.images + d.factors + 2 * d.local + d.maps + 256;
}

fi_status fi_delta_forward(const fi_delta_desc *desc, const void *q, const void *k, const void *v, const float *decay,
                           const float *beta, const float *state, const int32_t *lengths, void *y, float *final,
                           void *saved, void *workspace, void *stream) {
    static const char *call = "fi_delta_forward";
    if (const char *why = delta_check(desc)) return op_fail(FI_EINVAL, call, why);
    const bool steps = desc->T == 0 || (desc->T <= kDeltaSteps && !saved);
    const size_t es = value_bytes(desc->dtype);
    if (desc->T > 0 && (!q || !k || !v || !decay || !beta || !y || (!steps && !workspace)))
        return op_fail(FI_EINVAL, call, "q, k, v, decay, beta, y and the workspace are required");
    if (!aligned(es, {q, k, v, y}) || !aligned(4, {decay, beta, state, lengths, final}) || !aligned(256, {saved, workspace}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const DeltaPlan d = delta_plan(desc);
    DeltaArgs a = {};
    delta_args(desc, d, a);
    const int64_t rows = a.T * a.B;
    const size_t qk = (size_t)a.HK * a.dk * es, vb = (size_t)a.H * a.dv * es, hb = (size_t)a.H * 4;
    const size_t sb = (size_t)a.B * a.H * a.dk * a.dv * 4, lb = (size_t)a.B * 4;
    const size_t sv = fi_delta_saved_bytes(desc), ws = fi_delta_workspace_bytes(desc, 0);
    const View vstate = {state, 1, sb, sb}, vfinal = {final, 1, sb, sb};
    const View out[] = {vfinal, {y, rows, vb, (size_t)a.ldy * es}, {saved, 1, sv, sv}, {steps ? nullptr : workspace, 1, ws, ws}};
    const View in[] = {{q, rows, qk, (size_t)a.ldq * es}, {k, rows, qk, (size_t)a.ldk * es}, {v, rows, vb, (size_t)a.ldv * es},
                       {decay, rows, hb, (size_t)a.ldg * 4}, {beta, rows, hb, (size_t)a.ldb * 4}, {lengths, 1, lb, lb}};
    const bool inplace = final && state == final;
    if (outputs_meet(out, 4, in, 6) || outputs_meet(out + 1, 3, &vstate, 1) || (!inplace && views_meet(vfinal, vstate)))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    a.q = q, a.k = k, a.v = v, a.g = decay, a.beta = beta, a.state = state, a.lengths = lengths, a.y = y, a.final = final;
    char *w = (char *)workspace;
    a.images = w, w += d.images;
    a.factors = (float *)w, w += d.factors;
    a.starts = (float *)w, w += d.local;
    a.local = (float *)w, w += d.local;
    a.mapst = (float *)w;
    if (saved) {
        char *s = (char *)saved;
        a.states = (float *)s, s += d.states;
        a.w = (float *)s, s += d.rows;
        a.maps = (float *)s;
    }
    const hipStream_t st = (hipStream_t)stream;
    if (a.T == 0 && !final && !saved) return FI_OK;
    if (desc->dtype == FI_F32) forward<float>(a, d, steps, st);
    else if (desc->dtype == FI_BF16) forward<bf16_t>(a, d, steps, st);
    else forward<f16_t>(a, d, steps, st);
    return op_launched(call);
}

}  // extern "C"
