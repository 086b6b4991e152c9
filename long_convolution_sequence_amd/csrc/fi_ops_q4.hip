// Matrix-vector products with 4-bit weights and group scales (fi_q4_*).
//
// On the matrix units: a wave takes 16 outputs and steps of 32 inputs
// (v_mfma_f32_16x16x32, weights as A, the rows of x as columns of B).  A code
// becomes a 16-bit float without arithmetic: its four bits go to the top of the
// significand of 16.0, which gives 16 + code exactly; a second product into the
// same sum, with -(16 + zero) made in the same way along the whole row of A, takes
// the zeros away.  bf16 and fp16 inputs multiply as they are; fp32 inputs are cut
// into three bf16 terms (8 significand bits each, by truncation, so the terms add
// up to x exactly), each a column of its own.
//
// What bounds it: the bytes of the codes at the large sizes (28672 x 8192 bf16 in
// groups of 128, zeros: 28.5 us, 4.3 TB/s; in groups of 32 36 us, with the scales'
// conversions), a wave's chain of loads, products and the join at the small ones
// (5003 x 4999 fp16 of 16 rows 12 us, 2592 x 864 fp32 of 8 rows 5 us).  A workgroup
// takes 16 outputs, its waves split K (128 inputs a step, a step a wave in turn).  A
// wave brings x of its step through LDS into the order of the product's operand (read
// from memory in that order, 31 us where this takes 12); with many outputs it takes
// two or four row tiles for each operand.  The waves' sums meet in LDS, in their
// order.  More steps' loads ahead, or codes read as streams: no faster.
//
// Layout of the packed weights, tiles of 16 outputs x 128 inputs:
//   codes  [N/16][K/128][64 lanes][4 words]   lane l: output l & 15; word s holds
//          the inputs 32 s + 8 (l >> 4) + 0..7: value 2p in bits 4p..4p+3, value
//          2p + 1 in bits 16 + 4p..
//   scales [N/16][K/128][4][groups][4]: a lane of the product holds the outputs
//          (l >> 4) * 4 + 0..3, and reads their scales of all the step's groups
//          (128 / group) side by side
//   zeros  [N/16][K/128][16 outputs][groups] of 4 bits, as the lanes of A need them
// with N and K rounded up (codes 0, scales 0).
#include <type_traits>

#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kQ4MaxRows = 16;
constexpr int kQ4Max = 1 << 20;

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f16x8 = __attribute__((ext_vector_type(8))) _Float16;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) unsigned;

struct Q4Layout {
    int tiles, kt, groups;         // row tiles, 128-wide steps, groups of the padded K
    size_t codes, scales, zeros, total;   // byte offsets
};

bool q4_layout(const fi_q4_desc *q, Q4Layout &l) {
    l.tiles = (q->N + 15) / 16;
    l.kt = (q->K + 127) / 128;
    l.groups = l.kt * (128 / q->group);
    l.codes = 0;
    l.scales = (size_t)l.tiles * l.kt * 1024;
    l.zeros = l.scales + up256((size_t)l.tiles * l.groups * 16 * value_bytes(q->scale_dtype));
    l.total = l.zeros + (q->has_zeros ? up256((size_t)l.tiles * l.groups * 8) : 0);
    return true;
}

const char *q4_check(const fi_q4_desc *q) {
    if (!q) return "null descriptor";
    if (q->N < 1 || q->N > kQ4Max || q->K < 1 || q->K > kQ4Max) return "N and K are not in 1 .. 2^20";
    if (q->group != 32 && q->group != 64 && q->group != 128) return "group is not 32, 64 or 128";
    if (!value_type(q->scale_dtype)) return "scale_dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->has_zeros != 0 && q->has_zeros != 1) return "has_zeros is not 0 or 1";
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    return nullptr;
}

// The laying out and the quantizing run once a weight; their threads go through
// the whole of it in strides (a launch has less than 2^32 threads).
// One word of codes per thread and turn.
__global__ void __launch_bounds__(256) k_q4_codes(int N, int K, int kt, const uint8_t *codes, unsigned *out,
                                                  int64_t words) {
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < words; i += gridDim.x * (int64_t)256) {
        const int s = i & 3, lane = (i >> 2) & 63;
        const int64_t tile = i >> 8;
        const int n = (int)(tile / kt) * 16 + (lane & 15);
        const int k0 = (int)(tile % kt) * 128 + s * 32 + (lane >> 4) * 8;
        const uint8_t *from = codes + (size_t)n * K + k0;
        Chunk<uint8_t, 8> q = (Chunk<uint8_t, 8>)(uint8_t)0;
        if (n < N && k0 + 8 <= K)
            q = *reinterpret_cast<const Chunk<uint8_t, 8> *>(from);
        else if (n < N)
            for (int j = 0; j < 8; ++j) q[j] = k0 + j < K ? from[j] : 0;
        unsigned w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) w |= (q[j] & 15u) << ((j >> 1) * 4 + (j & 1) * 16);
        out[i] = w;
    }
}

// Where value i of the scales' layout comes from: its output and its group.
struct Q4Where {
    int n, g;
    __device__ __forceinline__ Q4Where(int64_t i, int kt, int per) {
        const int row = (int)(i & 3), in = (int)((i >> 2) % per), kq = (int)((i >> 2) / per & 3);
        const int64_t step = i / (16 * per);
        n = (int)(step / kt) * 16 + kq * 4 + row;
        g = (int)(step % kt) * per + in;
    }
};

template <typename V>
__global__ void __launch_bounds__(256) k_q4_scales(int N, int have, int kt, int per, const V *scales, V *out,
                                                   int64_t n) {
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += gridDim.x * (int64_t)256) {
        const Q4Where w(i, kt, per);
        out[i] = w.n < N && w.g < have ? scales[(size_t)w.n * have + w.g] : (V)0.f;
    }
}

// Four zeros per value: outputs in order, the groups of a step inside an output.
__global__ void __launch_bounds__(256) k_q4_zeros(int N, int have, int kt, int per, const uint8_t *zeros,
                                                  uint16_t *out, int64_t n) {
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += gridDim.x * (int64_t)256) {
        unsigned v = 0;
        for (int j = 0; j < 4; ++j) {
            const int64_t at = (i * 4 + j) / per, step = at / 16;
            const int w = (int)(step / kt) * 16 + (int)(at % 16), g = (int)(step % kt) * per + j % per;
            if (w < N && g < have) v |= (zeros[(size_t)w * have + g] & 15u) << (4 * j);
        }
        out[i] = (uint16_t)v;
    }
}

// One group of one row per wave and turn.
template <typename W, typename S>
__global__ void __launch_bounds__(256) k_q4_quantize(int N, int K, int group, int have, const W *w, int64_t ldw,
                                                     uint8_t *codes, S *scales) {
    const int lane = threadIdx.x & 63;
    const int64_t groups = (int64_t)N * have;
    for (int64_t i = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6); i < groups; i += gridDim.x * (int64_t)4) {
        const int n = (int)(i / have), g = (int)(i - (int64_t)n * have);
        const int k0 = g * group, k1 = k0 + group < K ? k0 + group : K;
        float m = 0.f;
        for (int k = k0 + lane; k < k1; k += 64) m = fmaxf(m, fabsf((float)w[n * ldw + k]));
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
        const S s = (S)(m / 7.f);
        const float f = (float)s;
        for (int k = k0 + lane; k < k1; k += 64) {
            float q = 0.f;
            if (f > 0.f) q = fminf(fmaxf(rintf((float)w[n * ldw + k] / f), -7.f), 7.f);
            codes[(size_t)n * K + k] = (uint8_t)(8 + (int)q);
        }
        if (lane == 0) scales[i] = s;
    }
}

struct Q4Args {
    const u32x4 *codes;
    const void *scales;
    const uint8_t *zeros;      // or NULL
    const void *x;
    void *y;
    int64_t ldx, ldy;
    int N, K, kt, rows;
    int cols;                  // columns of the product: rows x terms
};

// What x of a type becomes in the product: its terms, and the operands' type.
template <typename V> struct Operand;
template <> struct Operand<bf16_t> {
    static constexpr int terms = 1;
    using T = bf16_t;
    using X8 = bf16x8;
};
template <> struct Operand<f16_t> {
    static constexpr int terms = 1;
    using T = f16_t;
    using X8 = f16x8;
};
template <> struct Operand<float> {
    static constexpr int terms = 3;
    using T = bf16_t;
    using X8 = bf16x8;
};

__device__ __forceinline__ f32x4 product(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 product(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16 + code of a word's eight codes.
__device__ __forceinline__ void weights(unsigned w, bf16x8 &out) {
    union {
        unsigned u[4];
        bf16x8 v;
    } r;
    r.u[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    r.u[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    r.u[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    r.u[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    out = r.v;
}
__device__ __forceinline__ void weights(unsigned w, f16x8 &out) {
    union {
        unsigned u[4];
        f16x8 v;
    } r;
    r.u[0] = ((w << 6) & 0x03c003c0u) | 0x4c004c00u;
    r.u[1] = ((w << 2) & 0x03c003c0u) | 0x4c004c00u;
    r.u[2] = ((w >> 2) & 0x03c003c0u) | 0x4c004c00u;
    r.u[3] = ((w >> 6) & 0x03c003c0u) | 0x4c004c00u;
    out = r.v;
}

// -(16 + zero) eight times; -24 where no zeros are given.
__device__ __forceinline__ void minus(unsigned zero, bf16x8 &out) {
    const unsigned z = zero << 19 | zero << 3 | 0xc180c180u;
    const u32x4 v = {z, z, z, z};
    out = __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ void minus(unsigned zero, f16x8 &out) {
    const unsigned z = zero << 22 | zero << 6 | 0xcc00cc00u;
    const u32x4 v = {z, z, z, z};
    out = __builtin_bit_cast(f16x8, v);
}

// Eight inputs k.. of a row of x, zeros from K on.
template <typename V>
__device__ __forceinline__ Chunk<V, 8> inputs(const V *row, int k, int K) {
    if (k + 8 <= K) return *reinterpret_cast<const Chunk<V, 8> *>(row + k);
    Chunk<V, 8> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? row[k + i] : (V)0.f;
    return v;
}

// The three bf16 terms of fp32 values: eight significand bits each, by
// truncation; the last one needs no cut.
__device__ __forceinline__ void cut(float v, bf16_t &hi, bf16_t &mid, bf16_t &lo) {
    const float h = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    v -= h;
    const float m = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    hi = (bf16_t)h;
    mid = (bf16_t)m;
    lo = (bf16_t)(v - m);
}

// Eight inputs of a row into LDS, at its columns of a chunk's [column].
template <typename V, typename X8>
__device__ __forceinline__ void put(X8 *to, const Chunk<V, 8> &v) {
    if constexpr (Operand<V>::terms == 1) {
        X8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = v[j];
        to[0] = o;
    } else {
        X8 o[3];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bf16_t t[3];
            cut(v[j], t[0], t[1], t[2]);
            o[0][j] = t[0], o[1][j] = t[1], o[2][j] = t[2];
        }
        to[0] = o[0], to[1] = o[1], to[2] = o[2];
    }
}

constexpr int kQ4Waves = 16;           // waves of a workgroup at most
constexpr int kQ4Lds = 64 * 1024;      // bytes of LDS at most
// Row tiles of a wave where there are kQ4TallFrom of them.  Four save more of x's
// way through LDS, two leave registers for more waves, which the groups' scales
// want: 28672 x 8192 bf16 in groups of 128 28.6 us with four, 29.6 with two; in
// groups of 32 41 and 36.5; 13757 x 14352 (860 row tiles) in groups of 32 41 with
// one, 32 with two; 9258 x 13611 fp32 (579) 30 with one, 34.5 with two.
constexpr int kQ4TallFrom = 768;
template <int GROUP> constexpr int kQ4Tall = GROUP == 128 ? 4 : 2;

// RT row tiles and CT column tiles of 16.  Every wave brings x of its step into
// a part of LDS of its own, so nothing waits at a barrier before the end.
template <typename V, typename S, int GROUP, int CT, int RT>
__global__ void __launch_bounds__(RT > 1 ? 512 : kQ4Waves * 64) k_q4(Q4Args p) {
    using Op = Operand<V>;
    using X8 = typename Op::X8;
    constexpr int TERMS = Op::terms, PER = 128 / GROUP;
    constexpr int ROWS = TERMS == 1 ? 16 : CT * 16 / TERMS;      // rows of x at most
    constexpr int LOADS = (ROWS + 3) / 4;                        // 16 lanes read a row's step
    using Scales = S __attribute__((ext_vector_type(4 * PER)));
    using Zeros = std::conditional_t<PER == 4, uint16_t, uint8_t>;     // an output's, or two outputs'
    const Scales *scales = static_cast<const Scales *>(p.scales);
    const Zeros *zeros = reinterpret_cast<const Zeros *>(p.zeros);
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int col = lane & 15, kq = lane >> 4;
    const int nibble = PER == 1 ? lane % 2 * 4 : 0;
    const int64_t tile = blockIdx.x * (int64_t)RT;
    const int last = (p.N + 15) / 16 - 1;
    // an odd number of 16-byte places between chunks: at an even one the writes of
    // x (a row's chunks from 16 lanes) would meet in few banks
    const int pitch = p.cols | 1;
    X8 *xs = reinterpret_cast<X8 *>(lds) + wave * 16 * pitch;
    // this lane's column of each column tile (one without a column reads another's)
    int at[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) at[c] = kq * pitch + (c * 16 + col < p.cols ? c * 16 + col : 0);
    f32x4 y[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) y[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int u = wave; u < p.kt; u += waves) {
        u32x4 w[RT];
        Scales sc[RT];
        Zeros ze[RT];
        Chunk<V, 8> raw[LOADS];
#pragma unroll
        for (int m = 0; m < LOADS; ++m) {
            if (m * 4 >= p.rows) break;
            const int r = m * 4 + kq < p.rows ? m * 4 + kq : p.rows - 1;
            const V *x = static_cast<const V *>(p.x) + r * p.ldx;
            if (u * 128 + 128 <= p.K)
                raw[m] = *reinterpret_cast<const Chunk<V, 8> *>(x + u * 128 + col * 8);
            else
                raw[m] = inputs<V>(x, u * 128 + col * 8, p.K);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            // a row tile past the last one reads that one, and is not stored
            const int64_t at = (tile + r < last ? tile + r : last) * p.kt + u;
            w[r] = p.codes[at * 64 + lane];
            sc[r] = scales[at * 4 + kq];
            ze[r] = zeros ? zeros[PER == 1 ? at * 8 + col / 2 : at * 16 + col] : (Zeros)0x8888;
        }
        // [32-wide step][4][column]; a wave's LDS accesses are done in order, so the
        // reads of the step before come first
#pragma unroll
        for (int m = 0; m < LOADS; ++m)
            if (m * 4 + kq < p.rows) put<V>(xs + col * pitch + (m * 4 + kq) * TERMS, raw[m]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int g = 0; g < PER; ++g) {
            f32x4 acc[RT][CT];
            X8 less[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                minus(ze[r] >> (4 * g + nibble) & 15u, less[r]);
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int s = 0; s < GROUP / 32; ++s) {
                const int s32 = g * (GROUP / 32) + s;
                X8 b[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) b[c] = xs[s32 * 4 * pitch + at[c]];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    X8 q;
                    weights(w[r][s32], q);
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[r][c] = product(less[r], b[c], acc[r][c]);
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[r][c] = product(q, b[c], acc[r][c]);
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float scale = (float)sc[r][4 * g + i];
#pragma unroll
                    for (int c = 0; c < CT; ++c) y[r][c][i] = fmaf(scale, acc[r][c][i], y[r][c][i]);
                }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the waves' sums, in their order; then an input's terms, the smallest first
    float *part = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[((wave * CT + c) * 16 + kq * 4 + i) * 17 + col] = y[r][c][i];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * p.rows; i += blockDim.x) {
            const int n = i & 15, b = i >> 4;
            float v = 0.f;
#pragma unroll
            for (int j = TERMS - 1; j >= 0; --j) {
                const int k = b * TERMS + j;
                float q = 0.f;
                for (int u = 0; u < waves; ++u) q += part[((u * CT + (k >> 4)) * 16 + n) * 17 + (k & 15)];
                v += q;
            }
            if ((tile + r) * 16 + n < p.N) static_cast<V *>(p.y)[b * p.ldy + (tile + r) * 16 + n] = (V)v;
        }
    }
}

// Waves that split K: enough that the whole device has sixteen a CU (twice that
// with two row tiles a wave: 36.5 us against 55 at 28672 x 8192 in groups of 32; with
// one, 50 against 57 at 13757 x 14352), four at least, no more than there are steps.
int q4_waves(int groups, int kt, int rt, int most) {
    const int want = ((rt == 2 ? 8192 : 4096) + groups - 1) / groups;
    return std::min(std::min(std::max(want, 4), most), kt);
}

// With several column tiles a CU has registers for sixteen waves and LDS for few: a
// count that leaves part of either unused, and workgroups for a second round, goes
// down to the multiple of four with which more of them fit (7357 x 15788 of 8 fp32
// rows nine waves 43 us, eight 33; 9000 x 9000 of 16 five 54, four 44).  What bounds
// them then: the products, three terms' and the zeros' (13 and 9 us by the bytes);
// with fp32 scales in groups of 32 or 64 and three column tiles 6 or 2 registers
// spill besides.
int q4_fitting(int waves, int groups, int step) {
    const auto on_cu = [&](int w) { return std::min(16 / w, 160 * 1024 / (w * step)); };
    if (groups <= 256 * on_cu(waves)) return waves;
    for (int w = waves / 4 * 4; w >= 4 && w < waves; w -= 4)
        if (on_cu(w) > on_cu(waves)) return w;
    return waves;
}

template <typename V, typename S, int GROUP, int CT, int RT>
void q4_launch(const Q4Args &a, hipStream_t st) {
    const int tiles = (a.N + 15) / 16, groups = (tiles + RT - 1) / RT;
    const size_t step = (size_t)(a.cols | 1) * 256;      // bytes of x of one step in LDS
    int waves = std::min(q4_waves(groups, a.kt, RT, RT > 1 ? 8 : kQ4Waves), kQ4Lds / (int)step);
    if (CT > 1 && RT == 1 && waves % 4) waves = q4_fitting(waves, groups, (int)step);
    const size_t part = (size_t)waves * CT * 16 * 17 * sizeof(float);
    hipLaunchKernelGGL((k_q4<V, S, GROUP, CT, RT>), dim3((unsigned)groups), dim3(waves * 64),
                       std::max(waves * step, part), st, a);
}

template <typename V, typename S, int GROUP, int CT>
void q4_launch(const Q4Args &a, hipStream_t st) {
    if ((a.N + 15) / 16 >= kQ4TallFrom) q4_launch<V, S, GROUP, CT, kQ4Tall<GROUP>>(a, st);
    else q4_launch<V, S, GROUP, CT, 1>(a, st);
}

template <typename V, typename S, int GROUP>
void q4_launch(Q4Args a, hipStream_t st) {
    a.cols = a.rows * Operand<V>::terms;
    const int tiles = (a.cols + 15) / 16;
    if (tiles == 1) q4_launch<V, S, GROUP, 1>(a, st);
    if constexpr (Operand<V>::terms == 3) {
        if (tiles == 2) q4_launch<V, S, GROUP, 2>(a, st);
        if (tiles == 3) q4_launch<V, S, GROUP, 3>(a, st);
    }
}

template <typename V, typename S>
void q4_launch(const Q4Args &a, int group, hipStream_t st) {
    if (group == 32) q4_launch<V, S, 32>(a, st);
    else if (group == 64) q4_launch<V, S, 64>(a, st);
    else q4_launch<V, S, 128>(a, st);
}

template <typename V>
void q4_launch(const Q4Args &a, int group, int sdt, hipStream_t st) {
    if (sdt == FI_F32) q4_launch<V, float>(a, group, st);
    else if (sdt == FI_BF16) q4_launch<V, bf16_t>(a, group, st);
    else q4_launch<V, f16_t>(a, group, st);
}

// Workgroups of four waves for n pieces of work, `per` in one: eight a CU at most.
unsigned blocks(int64_t n, int per) { return (unsigned)std::min<int64_t>((n + per - 1) / per, 2048); }

template <typename W>
void quantize(const fi_q4_desc *q, int have, const void *w, int64_t ldw, uint8_t *codes, void *scales,
              hipStream_t st) {
    const dim3 grid(blocks((int64_t)q->N * have, 4)), wg(256);
    if (q->scale_dtype == FI_F32)
        hipLaunchKernelGGL((k_q4_quantize<W, float>), grid, wg, 0, st, q->N, q->K, q->group, have, (const W *)w,
                           ldw, codes, (float *)scales);
    else if (q->scale_dtype == FI_BF16)
        hipLaunchKernelGGL((k_q4_quantize<W, bf16_t>), grid, wg, 0, st, q->N, q->K, q->group, have, (const W *)w,
                           ldw, codes, (bf16_t *)scales);
    else
        hipLaunchKernelGGL((k_q4_quantize<W, f16_t>), grid, wg, 0, st, q->N, q->K, q->group, have, (const W *)w,
                           ldw, codes, (f16_t *)scales);
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_q4_packed_bytes(const fi_q4_desc *desc) {
    Q4Layout l;
    return !q4_check(desc) && q4_layout(desc, l) ? l.total : 0;
}

fi_status fi_q4_pack(const fi_q4_desc *desc, const uint8_t *codes, const void *scales, const uint8_t *zeros,
                     void *packed, void *stream) {
    static const char *call = "fi_q4_pack";
    if (const char *why = q4_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (!codes || !scales || !packed || (uintptr_t)packed % 256)
        return op_fail(FI_EINVAL, call, "codes, scales and packed (aligned to 256 bytes) are required");
    if (!aligned(value_bytes(desc->scale_dtype), {scales})) return op_fail(FI_EINVAL, call, "scales is not aligned to its values");
    if ((zeros != nullptr) != (desc->has_zeros != 0)) return op_fail(FI_EINVAL, call, "zeros do not go with has_zeros");
    Q4Layout l;
    q4_layout(desc, l);
    const int have = (desc->K + desc->group - 1) / desc->group;
    const size_t nk = (size_t)desc->N * desc->K, ns = (size_t)desc->N * have;
    const size_t sb = ns * value_bytes(desc->scale_dtype);
    const View out = {packed, 1, l.total, l.total};
    const View in[] = {{codes, 1, nk, nk}, {scales, 1, sb, sb}, {zeros, 1, ns, ns}};
    if (outputs_meet(&out, 1, in, 3)) return op_fail(FI_EINVAL, call, "packed shares memory with another argument");
    const hipStream_t st = (hipStream_t)stream;
    char *to = (char *)packed;
    const int64_t words = (int64_t)l.tiles * l.kt * 256, sc = (int64_t)l.tiles * l.groups * 16;
    hipLaunchKernelGGL(k_q4_codes, dim3(blocks(words, 256)), dim3(256), 0, st, desc->N, desc->K, l.kt, codes,
                       (unsigned *)(to + l.codes), words);
    if (desc->scale_dtype == FI_F32)
        hipLaunchKernelGGL((k_q4_scales<float>), dim3(blocks(sc, 256)), dim3(256), 0, st, desc->N, have, l.kt, 128 / desc->group,
                           (const float *)scales, (float *)(to + l.scales), sc);
    else    // both 16-bit types are copied as they are
        hipLaunchKernelGGL((k_q4_scales<bf16_t>), dim3(blocks(sc, 256)), dim3(256), 0, st, desc->N, have, l.kt, 128 / desc->group,
                           (const bf16_t *)scales, (bf16_t *)(to + l.scales), sc);
    if (zeros)
        hipLaunchKernelGGL(k_q4_zeros, dim3(blocks(sc / 4, 256)), dim3(256), 0, st, desc->N, have, l.kt,
                           128 / desc->group, zeros,
                           (uint16_t *)(to + l.zeros), sc / 4);
    return op_launched(call);
}

fi_status fi_q4_quantize(const fi_q4_desc *desc, int w_dtype, const void *w, int64_t ld_w, uint8_t *codes,
                         void *scales, void *stream) {
    static const char *call = "fi_q4_quantize";
    if (const char *why = q4_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (desc->has_zeros) return op_fail(FI_EINVAL, call, "has_zeros: the codes are symmetric about 8");
    if (!value_type(w_dtype)) return op_fail(FI_EINVAL, call, "w_dtype is none of FI_F32, FI_BF16, FI_F16");
    if (!w || !codes || !scales) return op_fail(FI_EINVAL, call, "w, codes and scales are required");
    const int64_t ldw = ld_w ? ld_w : desc->K;
    if (ldw < desc->K || ldw > (int64_t(1) << 40)) return op_fail(FI_EINVAL, call, "the row pitch is less than K");
    const int have = (desc->K + desc->group - 1) / desc->group;
    const size_t nk = (size_t)desc->N * desc->K, sb = (size_t)desc->N * have * value_bytes(desc->scale_dtype);
    const View out[] = {{codes, 1, nk, nk}, {scales, 1, sb, sb}};
    const size_t ws = value_bytes(w_dtype);
    if (!aligned(ws, {w}) || !aligned(value_bytes(desc->scale_dtype), {scales}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const View in = {w, desc->N, desc->K * ws, ldw * ws};
    if (outputs_meet(out, 2, &in, 1)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    const hipStream_t st = (hipStream_t)stream;
    if (w_dtype == FI_F32) quantize<float>(desc, have, w, ldw, codes, scales, st);
    else if (w_dtype == FI_BF16) quantize<bf16_t>(desc, have, w, ldw, codes, scales, st);
    else quantize<f16_t>(desc, have, w, ldw, codes, scales, st);
    return op_launched(call);
}

fi_status fi_q4_matvec(const fi_q4_desc *desc, const void *packed, int rows, int dtype, const void *x, int64_t ld_x,
                       void *y, int64_t ld_y, void *stream) {
    static const char *call = "fi_q4_matvec";
    if (const char *why = q4_check(desc)) return op_fail(FI_EINVAL, call, why);
    if (!value_type(dtype)) return op_fail(FI_EINVAL, call, "dtype is none of FI_F32, FI_BF16, FI_F16");
    if (rows < 1 || rows > kQ4MaxRows) return op_fail(FI_EINVAL, call, "rows is not in 1 .. 16");
    if (!packed || !x || !y || (uintptr_t)packed % 256)
        return op_fail(FI_EINVAL, call, "packed (aligned to 256 bytes), x and y are required");
    Q4Args a = {};
    a.ldx = ld_x ? ld_x : desc->K;
    a.ldy = ld_y ? ld_y : desc->N;
    if (a.ldx < desc->K || a.ldy < desc->N || a.ldx > (int64_t(1) << 40) || a.ldy > (int64_t(1) << 40))
        return op_fail(FI_EINVAL, call, "a row pitch is less than the row");
    Q4Layout l;
    q4_layout(desc, l);
    const size_t es = value_bytes(dtype);
    if (!aligned(es, {x, y})) return op_fail(FI_EINVAL, call, "x or y is not aligned to its values");
    const View out = {y, rows, desc->N * es, a.ldy * es};
    const View in[] = {{x, rows, desc->K * es, a.ldx * es}, {packed, 1, l.total, l.total}};
    if (outputs_meet(&out, 1, in, 2)) return op_fail(FI_EINVAL, call, "y shares memory with another argument");
    a.codes = (const u32x4 *)((const char *)packed + l.codes);
    a.scales = (const char *)packed + l.scales;
    a.zeros = desc->has_zeros ? (const uint8_t *)packed + l.zeros : nullptr;
    a.x = x, a.y = y, a.N = desc->N, a.K = desc->K, a.kt = l.kt, a.rows = rows;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FI_F32) q4_launch<float>(a, desc->group, desc->scale_dtype, st);
    else if (dtype == FI_BF16) q4_launch<bf16_t>(a, desc->group, desc->scale_dtype, st);
    else q4_launch<f16_t>(a, desc->group, desc->scale_dtype, st);
    return op_launched(call);
}

}  // extern "C"
