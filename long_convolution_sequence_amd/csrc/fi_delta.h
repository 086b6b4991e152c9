// The gated delta rule: what its kernels share.  Per head, with decays a = e^g:
//   S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  y_t = scale S_t^T q_t.
// A chunk of C positions at once: with G the sum of g from the chunk's start,
// E_ij = e^(G_i - G_j) and S the state before the chunk,
//   (I + A) w = v - e^G K S,  A_ij = E_ij (k_i . k_j) b_j (i > j),
//   y = scale (e^G Q S + (E o Q K^T)(b w)),  S' = e^(G_C) S + sum_j e^(G_C - G_j) k_j (b_j w_j)^T.
// Only S passes from chunk to chunk, and its columns do not meet: a wave runs 16 columns
// of a head along the sequence, with S in the accumulators of the matrix instruction
// v_mfma_f32_16x16x32_bf16 (the chains); what is a chunk's own runs for all chunks at
// once on v_mfma_f32_32x32x16_bf16.
//
// Operands.  An operand is kept in LDS or memory as an image of pieces of 1 KB, lane l's
// 16 bytes what the instruction takes of it.  Of 32 rows x 16 values of the summed index
// they are the values 8 (j / 4) + 4 (l / 32) + j % 4, j < 8, of row l % 32.  In that order
// of the summed index an accumulator (lane l: rows 8 (r / 4) + 4 (l / 32) + r % 4 of column
// l % 32) is an operand as it stands, registers 8 s .. 8 s + 7 its step s: what one product
// gives goes into the next without leaving the lane.  The chains' pieces (tile_at) do the
// same for 16 rows x 32 values.
//
// Values in 32 bits are multiplied as terms of bf16 (x = t0 + t1 + t2, each the
// rounding of what is left, exact to 2^-24): of two factors the products of terms i
// and j with i + j <= 2 are taken.  bf16 inputs are one term, fp16 two, fp32 three.
#pragma once
#include <type_traits>

#include "fi_ops.h"

namespace fi {

constexpr int kDeltaMaxK = 128;        // channels of a key at most
constexpr int kDeltaMaxV = 1024;       // of a value
constexpr float kDeltaUnit = 1e-6f;    // k / sqrt(sum k^2 + this)
constexpr int kPiece = 1024;           // bytes of an operand's piece
constexpr int kDeltaFactors = 16;      // floats a position, of which nine are used: whole pieces
constexpr float kLog2e = 1.44269504088896f;

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using bf16x4 = __bf16 __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using f32x4 = float __attribute__((ext_vector_type(4)));

// Terms of an input and positions of a chunk.  Chunks of fp16 and fp32 are 32 long: the
// images of two and three terms of 64 positions leave a CU one workgroup or none.
template <typename T>
struct DeltaType;
template <>
struct DeltaType<bf16_t> {
    static constexpr int terms = 1, chunk = 64;
};
template <>
struct DeltaType<f16_t> {
    static constexpr int terms = 2, chunk = 32;
};
template <>
struct DeltaType<float> {
    static constexpr int terms = 3, chunk = 32;
};
inline int delta_chunk(int dtype) { return dtype == FI_BF16 ? 64 : 32; }

struct DeltaArgs {
    const void *q, *k, *v, *dy;
    void *y, *dq, *dk_out, *dv_out;
    const float *g, *beta, *state, *dfinal;
    float *final, *dstate, *dg, *dbeta;
    const int32_t *lengths;
    int64_t T, chunks, per;                // positions, chunks, chunks of a segment
    int64_t ldq, ldk, ldv, ldg, ldb, ldy, lddy, lddq, lddk, lddv, lddg, lddb;
    int B, HK, H, dk, dv, segments;
    int unit;
    float scale;
    // [chunk][B][H] of each
    char *images;                          // M and P of a chunk (backwards N^T and P^T)
    float *factors;                        // [kDeltaFactors][C]
    float *states;                         // [dk][dv] before each chunk
    float *ends;                           // backwards [dk][dv] after each chunk
    float *w, *x;                          // [C][dv]
    // [segment][B][H]
    float *local;                          // [dk][dv] what a segment makes of nothing
    float *maps, *mapst;                   // [dk][dk] what it makes of a state, and its transpose
    float *starts;                         // [dk][dv] the state before it (backwards: the gradient behind it)
};

// Loads from LDS are not moved across: all at once they would spill.
__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }

// A number for the whole wave or a lane that the compiler takes for a new one: what is
// made of it (a chunk's offsets and masks, 32 registers each) is made where it is used
// and not kept from chunk to chunk.
template <typename I>
__device__ __forceinline__ I anew(I v) {
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ unsigned anew_lane(unsigned v) {
    asm volatile("" : "+v"(v));
    return v;
}

// ---- operands ------------------------------------------------------------------

template <int N>
struct Frag {
    bf16x8 t[N];
};

using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f32x2 = float __attribute__((ext_vector_type(2)));

// One term of two values, and what is left of them: x - t as the dot product
// t . (-1, 0) + x of bf16 pairs, exact, in one instruction a value (unpacking and
// subtracting take two).  The factors come from registers: as immediates of a packed
// instruction they would have to differ in their halves.
__device__ __forceinline__ bf16x2 term(float &x, float &y, bool more) {
    const bf16x2 t = __builtin_convertvector((f32x2{x, y}), bf16x2);
    if (more) {
        unsigned lo = 0x0000bf80u, hi = 0xbf800000u;
        asm("" : "+s"(lo));
        asm("" : "+s"(hi));
        x = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(bf16x2, lo), x, false);
        y = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(bf16x2, hi), y, false);
    }
    return t;
}

// Terms of eight values.
template <int N>
__device__ __forceinline__ Frag<N> split(const float (&x)[8]) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float u = x[i], v = x[i + 1];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const bf16x2 two = term(u, v, t + 1 < N);
            f.t[t][i] = two[0], f.t[t][i + 1] = two[1];
        }
    }
    return f;
}

// Step `s` (16 rows) of an accumulator as a right operand.
template <int N>
__device__ __forceinline__ Frag<N> step_of(const f32x16 &v, int s) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[s * 8 + i];
    return split<N>(x);
}

// acc += a b, the products of terms i and j with i + j <= ORDER.
template <int ORDER, int NA, int NB>
__device__ __forceinline__ void multiply(f32x16 &acc, const Frag<NA> &a, const Frag<NB> &b) {
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j <= ORDER) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[i], b.t[j], acc, 0, 0, 0);
}

// An image's piece as an operand; terms are `stride` bytes apart.
template <int N>
__device__ __forceinline__ Frag<N> piece(const char *image, int at, int stride) {
    Frag<N> f;
#pragma unroll
    for (int t = 0; t < N; ++t)
        f.t[t] = *reinterpret_cast<const bf16x8 *>(image + t * stride + at * kPiece + (threadIdx.x & 63) * 16);
    return f;
}

// Byte of value `k` of row `row` in an image with `steps` pieces along the summed
// index; four values from a multiple of four on are neighbours.
__device__ __forceinline__ int image_at(int row, int k, int steps) {
    return ((row >> 5) * steps + (k >> 4)) * kPiece + (((k >> 2) & 1) * 32 + (row & 31)) * 16 + ((k >> 3) & 1) * 8;
}

template <int N>
__device__ __forceinline__ void put_terms(char *image, int at, int stride, const float (&x)[4]) {
    float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const bf16x2 a = term(r[0], r[1], t + 1 < N), b = term(r[2], r[3], t + 1 < N);
        *reinterpret_cast<bf16x4 *>(image + t * stride + at) = bf16x4{a[0], a[1], b[0], b[1]};
    }
}
// Values that are their own term.
template <int N>
__device__ __forceinline__ void put_terms(char *image, int at, int, const bf16_t (&x)[4]) {
    *reinterpret_cast<bf16x4 *>(image + at) = bf16x4{x[0], x[1], x[2], x[3]};
}

// The chains' operands: v_mfma_f32_16x16x32_bf16, so that a wave takes 16 columns and
// four waves share a SIMD: what one waits for (a product that adds to the last, LDS,
// memory) runs under the others.  A piece is 16 rows x 32 values of the summed index,
// lane l's 16 bytes the values 16 (j / 4) + 4 (l / 16) + j % 4, j < 8, of row l % 16; an
// accumulator (lane l: rows 4 (l / 16) + r of column l % 16) is half a right operand.
__device__ __forceinline__ int tile_at(int row, int k, int steps) {
    return ((row >> 4) * steps + (k >> 5)) * kPiece + (((k >> 2) & 3) * 16 + (row & 15)) * 16 + ((k >> 4) & 1) * 8;
}
__device__ __forceinline__ int tile_row(int r) { return 4 * ((threadIdx.x >> 4) & 3) + r; }
template <int N, int M>
__device__ __forceinline__ Frag<N> step_of(const f32x4 (&v)[M], int s) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[2 * s][i], x[4 + i] = v[2 * s + 1][i];
    return split<N>(x);
}
template <int ORDER, int NA, int NB>
__device__ __forceinline__ void multiply(f32x4 &acc, const Frag<NA> &a, const Frag<NB> &b) {
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j <= ORDER) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.t[i], b.t[j], acc, 0, 0, 0);
}

// Row of register r of an accumulator, for the lane's half.
__device__ __forceinline__ int acc_row(int r) { return 8 * (r >> 2) + 4 * ((threadIdx.x >> 5) & 1) + (r & 3); }

// Four values of a row from d on, zeros behind D and where the row does not count
// (it is read all the same).  No lane branches: a load in a branch of its own would be
// waited for there.  VEC: D is a multiple of four.
template <bool VEC, typename T>
__device__ __forceinline__ void load4(float (&x)[4], const T *row, int d, int D, bool live) {
    if (VEC) {
        const Chunk<T, 4> v = *reinterpret_cast<const Chunk<T, 4> *>(row + min(d, D - 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = live && d < D ? (float)v[i] : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T v = row[min(d + i, D - 1)];
            x[i] = live && d + i < D ? (float)v : 0.f;
        }
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ Chunk<T, 4> raw4(const T *row, int d, int D) {
    if (VEC) return *reinterpret_cast<const Chunk<T, 4> *>(row + min(d, D - 4));
    Chunk<T, 4> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row[min(d + i, D - 1)];
    return v;
}

// C rows of a tensor on their way into images (TILES: of 16-row pieces): a thread takes
// four rows of four channels, with TILES one such block (chain_grid), else of 256 as many
// as it takes.  load() reads them ahead, rows from `live` (at least one) on and channels
// from D on as zeros; put() writes images: `rows` with the channels as the summed
// index, `cols` (the transpose) with the positions, either null.
template <typename T, int C, int DK, bool TILES>
struct Stage {
    static constexpr int N = DeltaType<T>::terms, RUNS = DK / 4, UNITS = C / 4 * RUNS, EACH = TILES ? 1 : (UNITS + 255) / 256;
    Chunk<T, 4> raw[EACH][4];

    template <bool VEC>
    __device__ __forceinline__ void load(const T *x, unsigned pitch, int D, int live) {
        const unsigned tid = anew_lane(threadIdx.x);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int u = e * (int)blockDim.x + (int)tid, i = u / RUNS * 4, d = u % RUNS * 4;
            if (u >= UNITS) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const unsigned row = min(i + r, live - 1) * pitch;
                if (VEC)
                    raw[e][r] = *reinterpret_cast<const Chunk<T, 4> *>(in_row(x, row + min(d, D - 4)));
                else
#pragma unroll
                    for (int j = 0; j < 4; ++j) raw[e][r][j] = *in_row(x, row + min(d + j, D - 1));
            }
        }
    }
    __device__ __forceinline__ void load(const T *x, unsigned pitch, int D, int live) {
        if ((D & 3) == 0) load<true>(x, pitch, D, live);
        else load<false>(x, pitch, D, live);
    }
    template <bool FULL>
    __device__ __forceinline__ void put(int D, int live, char *rows, char *cols) const {
        constexpr int IMAGE = C * DK * 2;
        using V = std::conditional_t<N == 1, T, float>;
        const unsigned tid = anew_lane(threadIdx.x);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int u = e * (int)blockDim.x + (int)tid, i = u / RUNS * 4, d = u % RUNS * 4;
            if (u >= UNITS) break;
            V m[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) m[r][j] = FULL || (i + r < live && d + j < D) ? (V)raw[e][r][j] : (V)0.f;
            if (rows) {
#pragma unroll
                for (int r = 0; r < 4; ++r) put_terms<N>(rows, TILES ? tile_at(i + r, d, DK / 32) : image_at(i + r, d, DK / 16), IMAGE, m[r]);
            }
            if (cols) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const V t[4] = {m[0][c], m[1][c], m[2][c], m[3][c]};
                    put_terms<N>(cols, TILES ? tile_at(d + c, i, C / 32) : image_at(d + c, i, C / 16), IMAGE, t);
                }
            }
        }
    }
    __device__ __forceinline__ void put(int D, int live, char *rows, char *cols) const {
        D = anew(D), live = anew(live);
        if (live == C && D == DK) put<true>(D, live, rows, cols);
        else put<false>(D, live, rows, cols);
    }
};

// Addresses below are an address for the whole wave and a 32-bit byte offset of the
// lane: a chunk's rows lie within 2^32 bytes (delta_check).

// A column of C rows in the places of accumulators, `at` for the whole wave.  Rows from
// `live` (at least one) on read the last one.
template <typename T, int M>
__device__ __forceinline__ void load_column(T (&v)[M][4], const T *at, unsigned column, unsigned pitch, int live) {
    column = anew_lane(column), pitch = anew(pitch), live = anew(live);
    if (live == M * 16) {
        const unsigned mine = column + tile_row(0) * pitch;
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[i][r] = *in_row(at, mine + (i * 16 + r) * pitch);
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[i][r] = *in_row(at, column + min(i * 16 + tile_row(r), live - 1) * pitch);
    }
}

// The way back: `rows` rows are there, those from `live` on get zeros.
template <typename T, int M>
__device__ __forceinline__ void store_column(T *at, unsigned column, unsigned pitch, const f32x4 (&v)[M], int rows, int live) {
    column = anew_lane(column), pitch = anew(pitch), live = anew(live), rows = anew(rows);
    if (live == M * 16) {
        const unsigned mine = column + tile_row(0) * pitch;
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) *in_row(at, mine + (i * 16 + r) * pitch) = (T)v[i][r];
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + tile_row(r);
                if (row < rows) *in_row(at, column + row * pitch) = (T)(row < live ? v[i][r] : 0.f);
            }
    }
}

// A state [dk][width] as accumulators and back; nothing lies past its edges.
template <int M>
__device__ __forceinline__ void load_state(f32x4 (&S)[M], const float *from, int dk, int width, int column) {
    const unsigned at = min(column, width - 1);
#pragma unroll
    for (int t = 0; t < M; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = t * 16 + tile_row(r);
            const float s = *in_row(from, at + (unsigned)(min(row, dk - 1) * width));
            S[t][r] = row < dk && column < width ? s : 0.f;
        }
}
template <int M>
__device__ __forceinline__ void store_state(float *to, const f32x4 (&S)[M], int dk, int width, int column) {
    if (column >= width) return;
    width = anew(width), dk = anew(dk), column = (int)anew_lane(column);
    const unsigned mine = column + tile_row(0) * width;
    if (dk == M * 16) {
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) *in_row(to, mine + (unsigned)((t * 16 + r) * width)) = S[t][r];
    } else {
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = t * 16 + tile_row(r);
                if (row < dk) *in_row(to, (unsigned)(column + row * width)) = S[t][r];
            }
    }
}

// Bytes (a multiple of 1 KB) from memory into LDS past the registers: each wave brings
// 1 KB at a time.  arrived() waits for this thread's share.
__device__ __forceinline__ void bring(char *to, const char *from, int bytes) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    for (int i = wave * kPiece; i < bytes; i += (int)(blockDim.x >> 6) * kPiece)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + i + lane * 16),
                                         (__attribute__((address_space(3))) void *)(to + i), 16, 0, 0);
}
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ int64_t delta_length(const DeltaArgs &p, int b) {
    if (!p.lengths) return p.T;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : n < p.T ? n : p.T;
}

__device__ __forceinline__ f32x16 zeros16() {
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    return v;
}

// ---- a chunk's own matrices ----------------------------------------------------

// Sum over a wave's lanes of the same half-position (lanes l and l ^ 32).
__device__ __forceinline__ float both_halves(float v) { return v + __shfl_xor(v, 32, 64); }

// A chunk's triangular matrices as images of 16-row pieces, those that hold zeros alone
// left out: of 64 positions, forwards (below the diagonal) rows 0 .. 31 have their first
// step alone, backwards (above it) rows 32 .. 63 their second.
template <int C>
constexpr int tri_pieces() { return C == 64 ? 6 : 2; }
template <int C, bool BACK>
__device__ __forceinline__ constexpr bool tri_in(int i, int s) { return C == 32 || (BACK ? i < 2 || s == 1 : i >= 2 || s == 0); }
template <int C, bool BACK>
__device__ __forceinline__ constexpr int tri_at(int i, int s) {
    return C == 32 ? i : BACK ? (i < 2 ? i * 2 + s : i + 2) : (i < 2 ? i : i * 2 - 2 + s);
}
// The factors that a chain reads, in whole pieces.
template <int C>
constexpr int factor_bytes() { return (5 * C * 4 + kPiece - 1) / kPiece * kPiece; }
template <typename T>
constexpr int image_bytes() { return tri_pieces<DeltaType<T>::chunk>() * kPiece * 6; }   // of a chunk: M and P in three terms

// A wave a chunk and head.  Forwards the images of M = (I + A)^-1 and of
// P_ij = scale E_ij (q_i . k_j) b_j, and the factors e^G_i of k_i S, scale e^G_i of
// q_i S, e^(G_C - G_i) b_i of k_i, e^(G_C).  Backwards those of N^T, N = (I + A')^-1
// with A'_ij = b_i E_ij (k_i . k_j), and of P^T without the b_j, and e^(G_C - G_i),
// scale e^G_i, e^G_i b_i, b_i, e^(G_C), both lengths' reciprocals and G in two floats.
// "unit" divides k and q by their lengths in these factors, so the operands stay the
// inputs themselves.
// The inverse: a lane solves for a column of a diagonal block of 32, row by row from
// registers, the rows of A read from LDS for all lanes of a block at once; the block
// below them is -N22 (A21 N11).  131072 positions of 9 heads of 96 bf16 268 us (1.2 GB
// moved, 250 at a copy's rate).
template <typename T, int KT, bool BACK, bool VEC>
__global__ void __launch_bounds__(64, DeltaType<T>::terms == 1 ? 2 : 1) k_delta_prep(DeltaArgs p) {
    constexpr int C = DeltaType<T>::chunk, N = DeltaType<T>::terms, MT = C / 32, CS = C / 16, KS = KT * 2, LD = C + 4;
    constexpr int MB = tri_pieces<C>() * kPiece;
    __shared__ __align__(16) float m[C * LD];
    __shared__ double sum[C];
    __shared__ float fb[C], fk[C], fq[C];
    const int lane = threadIdx.x, half = lane >> 5, col = lane & 31;
    const int64_t at = blockIdx.x;                       // [chunk][B][H]
    const int h = (int)(at % p.H), b = (int)(at / p.H % p.B), hk = h / (p.H / p.HK);
    const int64_t t0 = at / p.H / p.B * C, n = delta_length(p, b) - t0;
    if (n <= 0) return;
    const int live = n < C ? (int)n : C;

    // decays, in 64 bits: differences of sums keep their digits next to a large one
    if (lane < C) {
        const int64_t row = (t0 + min(lane, live - 1)) * p.B + b;
        float g = p.g[row * p.ldg + h], beta = p.beta[row * p.ldb + h];
        if (lane >= live) g = beta = 0.f;
        g = g < -1e4f ? -1e4f : g;                       // e^-10^4 is 0 in any case, -inf would be NaN in differences
        double s = (double)g * 1.4426950408889634;
#pragma unroll
        for (int d = 1; d < C; d *= 2) {
            const double o = __shfl_up(s, d, 64);
            if (lane >= d) s += o;
        }
        sum[lane] = s;
        fb[lane] = beta;
    }
    // k and q as operands, straight from memory: all of their loads together
    const T *k = static_cast<const T *>(p.k) + hk * p.dk, *q = static_cast<const T *>(p.q) + hk * p.dk;
    Chunk<T, 4> rawk[MT][KS][2], rawq[MT][KS][2];
    const auto fetch = [&](Chunk<T, 4> (&raw)[MT][KS][2], const T *from, int64_t ld) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const T *row = from + ((t0 + min(mt * 32 + col, live - 1)) * p.B + b) * ld;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) raw[mt][ks][e] = raw4<VEC>(row, ks * 16 + 4 * half + 8 * e, p.dk);
        }
    };
    fetch(rawk, k, p.ldk);
    fetch(rawq, q, p.ldq);
    float ssk[MT], ssq[MT];
    const auto operand = [&](const Chunk<T, 4> (&raw)[2], int mt, int ks, float &ss) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = mt * 32 + col < live && ks * 16 + 4 * half + 8 * (j >> 2) + (j & 3) < p.dk;
            x[j] = in ? (float)raw[j >> 2][j & 3] : 0.f;
            ss = fmaf(x[j], x[j], ss);
        }
        return split<N>(x);
    };
    Frag<N> ks_[MT][KS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        ssk[mt] = ssq[mt] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) ks_[mt][ks] = operand(rawk[mt][ks], mt, ks, ssk[mt]);
    }
    // A in rows (its upper half: zeros)
    {
        f32x16 kk[MT][MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) kk[i][j] = zeros16();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) multiply<2>(kk[i][j], ks_[i][ks], ks_[j][ks]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float a = both_halves(ssk[mt]);
            if (half == 0) fk[mt * 32 + col] = p.unit ? 1.f / sqrtf(a + kDeltaUnit) : 1.f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = i * 32 + acc_row(r), c = j * 32 + col;
                    m[row * LD + c] = j <= i && row > c ? exp2f((float)(sum[row] - sum[c])) * fk[c] * fk[row] * fb[BACK ? row : c] *
                                                              kk[i][j <= i ? j : 0][r]
                                                        : 0.f;
                }
    }
    // P in its registers
    f32x16 qk[MT][MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) qk[i][j] = zeros16();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const Frag<N> fq_ = operand(rawq[i][ks], i, ks, ssq[i]);
#pragma unroll
            for (int j = 0; j <= i; ++j) multiply<2>(qk[i][j], fq_, ks_[j][ks]);
        }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const float c = both_halves(ssq[mt]);
        if (half == 0) fq[mt * 32 + col] = p.unit ? 1.f / sqrtf(c + kDeltaUnit) : 1.f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = i * 32 + acc_row(r), c = j * 32 + col;
                const float e = row >= c ? exp2f((float)(sum[row] - sum[c])) * fk[c] : 0.f;
                qk[i][j][r] *= e * p.scale * fq[row] * (BACK ? 1.f : fb[c]);
            }
    __syncthreads();
    float x[32];
    const int block = MT == 2 ? half * 32 : 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float s0 = col == i ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(m + (block + i) * LD + block + j);
            s0 = fmaf(-a.x, x[j], s0);
            if (j + 1 < i) s1 = fmaf(-a.y, x[j + 1], s1);
            if (j + 2 < i) s2 = fmaf(-a.z, x[j + 2], s2);
            if (j + 3 < i) s3 = fmaf(-a.w, x[j + 3], s3);
        }
        x[i] = (s0 + s1) + (s2 + s3);
        if (i % 2) __builtin_amdgcn_sched_barrier(0);    // not all rows' loads at once: they would spill
    }
    __syncthreads();
    if (MT == 2 || half == 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i) m[(block + i) * LD + block + col] = x[i];
    }
    __syncthreads();
    if constexpr (MT == 2) {
        const auto rows = [&](int r0, int c0, int s) {   // a left operand of m
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = m[(r0 + col) * LD + c0 + s * 16 + 8 * (j >> 2) + 4 * half + (j & 3)];
            return split<3>(v);
        };
        f32x16 t = zeros16(), n21 = zeros16();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = m[(s * 16 + 8 * (j >> 2) + 4 * half + (j & 3)) * LD + col];
            multiply<2>(t, rows(32, 0, s), split<3>(v));
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) multiply<2>(n21, rows(32, 32, s), step_of<3>(t, s));
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; ++r) m[(32 + acc_row(r)) * LD + col] = -n21[r];
        __syncthreads();
    }
    const auto flush = [&](char *image) {                  // m (or its transpose) as an image
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
#pragma unroll
            for (int s = 0; s < C / 32; ++s) {
                if (!tri_in<C, BACK>(i, s)) continue;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = i * 16 + (lane & 15), c = s * 32 + 16 * (j >> 2) + 4 * (lane >> 4) + (j & 3);
                    v[j] = BACK ? m[c * LD + r] : m[r * LD + c];
                }
                const Frag<3> f = split<3>(v);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    *reinterpret_cast<bf16x8 *>(image + t * MB + tri_at<C, BACK>(i, s) * kPiece + lane * 16) = f.t[t];
            }
    };
    char *image = p.images + at * image_bytes<T>();
    flush(image);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) m[(i * 32 + acc_row(r)) * LD + j * 32 + col] = qk[i][j][r];
    __syncthreads();
    flush(image + 3 * MB);
    if (lane < C) {
        float *f = p.factors + at * kDeltaFactors * C;
        const float rise = exp2f((float)sum[lane]), fall = exp2f((float)(sum[C - 1] - sum[lane]));
        f[lane] = fk[lane] * (BACK ? fall : rise);
        f[C + lane] = p.scale * fq[lane] * rise;
        f[2 * C + lane] = fk[lane] * (BACK ? rise : fall) * fb[lane];
        f[3 * C + lane] = fb[lane];
        f[4 * C + lane] = exp2f((float)sum[C - 1]);
        f[5 * C + lane] = fk[lane];
        f[6 * C + lane] = fq[lane];
        f[7 * C + lane] = (float)sum[lane];
        f[8 * C + lane] = (float)(sum[lane] - (double)(float)sum[lane]);
    }
}

// ---- host side -----------------------------------------------------------------

constexpr int kDeltaWaves = 1536;      // sets of 32 columns that fill the card
constexpr int kDeltaLeast = 4;         // chunks of a segment at least

// Workgroups of a chain over `tiles` sets of 16 columns: up to eight waves each, as
// evenly as they go, and as many at least as bring a chunk's keys with a block of four
// rows x four channels a thread.
struct ChainGrid {
    unsigned groups, threads;
};
inline ChainGrid chain_grid(int tiles, int C, int KT) {
    const int groups = (tiles + 7) / 8, waves = (tiles + groups - 1) / groups;
    return {(unsigned)groups, (unsigned)std::max(64 * waves, C / 4 * KT * 8)};
}

struct DeltaPlan {
    int C, KT;
    int64_t chunks, per;               // chunks of the sequence, of a segment
    int segments;
    size_t images, factors, states, ends, rows, local, maps;   // bytes, each a multiple of 256
};

// Segments: a workgroup runs up to 128 columns of a head along the sequence; where that
// leaves most of the card idle, the sequence is cut into as many segments as fill it,
// each run once from nothing (with the columns of the state's own map, dk of them, beside
// it), joined, and run again from what is before it.  That is 2.5 times the work: with
// four segments a call over 2048 x 4 x 24 heads of 128 takes 437 us against 571 in one
// piece, over 4096 x 8 x 12 heads 798 against 1181, but with two 2048 x 8 x 24 heads 715
// against 705.  More segments than fill the card cost more to join (2.7 us each) than they
// bring (768, 1024, 1536, 2048 sets of columns: 131072 x 9 heads of 96 1627, 1777, 1650,
// 1750 us, 32768 x 6 heads of 128 607, 569, 603, 630).  At least four chunks a segment
// (two, four, eight, sixteen of them: 1024 x 9 heads of 96 88, 101, 160, 160 us, 4096 x 9
// heads 178, 149, 167, 261, 2048 x 4 heads of 128 fp32 168, 141, 164, 250, training pass
// over 1999 x 3 x 4 heads 72 x 41 fp16 345, 341, 388, 865).
inline DeltaPlan delta_plan(const fi_delta_desc *q) {
    DeltaPlan d = {};
    d.C = delta_chunk(q->dtype);
    d.KT = (q->dk + 31) / 32;
    d.chunks = (q->T + d.C - 1) / d.C;
    const int64_t heads = (int64_t)q->batch * q->heads, waves = heads * ((q->dv + 31) / 32);
    int64_t want = std::min<int64_t>(kDeltaWaves / std::max<int64_t>(1, waves), d.chunks / kDeltaLeast);
    if (want < 4) want = 1;
    d.per = std::max<int64_t>(1, (d.chunks + want - 1) / want);
    d.segments = (int)std::max<int64_t>(1, (d.chunks + d.per - 1) / d.per);
    const size_t all = (size_t)d.chunks * heads, C = d.C, sk = (size_t)q->dk * q->dv * 4;
    d.images = up256(all * (C == 64 ? tri_pieces<64>() : tri_pieces<32>()) * kPiece * 6);
    d.factors = up256(all * kDeltaFactors * C * 4);
    d.states = up256(all * sk);
    d.ends = up256(all * sk);
    d.rows = up256(all * C * q->dv * 4);
    const size_t parts = d.segments > 1 ? (size_t)d.segments * heads : 0;
    d.local = up256(parts * sk);
    d.maps = up256(parts * q->dk * q->dk * 4);
    return d;
}

const char *delta_check(const fi_delta_desc *q);
void delta_args(const fi_delta_desc *q, const DeltaPlan &plan, DeltaArgs &a);
// Joins the segments: starts[0] = first (or zeros), starts[s + 1] = maps[s] starts[s] + local[s];
// backwards from the last segment on, with the maps' transposes.
void delta_join(const DeltaArgs &a, const float *first, bool backward, hipStream_t st);

}  // namespace fi
