// Matrix-vector products with 4-bit weights and group scales (fi_q4_*).
//
// On the matrix units: a wave takes 16 outputs and steps of 32 inputs
// (v_mfma_f32_16x16x32_bf16, weights as A, the rows of x as columns of B).  A
// code becomes bf16 without arithmetic: its four bits go to the top of the
// significand of 16.0, which gives 16 + code exactly; the group's sum then
// loses (16 + zero) times the group's sum of x.  x in bf16 is one column; fp16
// and fp32 are cut into two and three bf16 terms (8 significand bits each, by
// truncation, so the terms add up to x exactly), each a column of its own.
//
// Layout of the packed weights, tiles of 16 outputs x 128 inputs of 1 KB:
//   codes  [N/16][K/128][64 lanes][4 words]   lane l: output l & 15; word s holds
//          the inputs 32 s + 8 (l >> 4) + 0..7: value 2p in bits 4p..4p+3, value
//          2p + 1 in bits 16 + 4p..
//   scales [N/16][groups][16], zeros [N/16][groups][16] in 4 bits
// with N and K rounded up (codes 0, scales 0); a lane of the product holds four
// outputs (l >> 4) * 4 + 0..3 and so reads four scales side by side.
#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kQ4MaxRows = 16;
constexpr int kQ4Max = 1 << 20;

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
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

// One word of codes per thread.
__global__ void __launch_bounds__(256) k_q4_codes(int N, int K, int kt, const uint8_t *codes, unsigned *out,
                                                  int64_t words) {
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (i >= words) return;
    const int s = i & 3, lane = (i >> 2) & 63;
    const int64_t tile = i >> 8;
    const int n = (int)(tile / kt) * 16 + (lane & 15);
    const int k0 = (int)(tile % kt) * 128 + s * 32 + (lane >> 4) * 8;
    unsigned w = 0;
    for (int j = 0; j < 8; ++j) {
        const unsigned q = n < N && k0 + j < K ? codes[(size_t)n * K + k0 + j] & 15u : 0u;
        w |= q << ((j >> 1) * 4 + (j & 1) * 16);
    }
    out[i] = w;
}

template <typename V>
__global__ void __launch_bounds__(256) k_q4_scales(int N, int have, int groups, const V *scales, V *out, int64_t n) {
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (i >= n) return;
    const int64_t tg = i >> 4;
    const int row = (int)(tg / groups) * 16 + (int)(i & 15), g = (int)(tg % groups);
    out[i] = row < N && g < have ? scales[(size_t)row * have + g] : (V)0.f;
}

__global__ void __launch_bounds__(256) k_q4_zeros(int N, int have, int groups, const uint8_t *zeros, uint16_t *out,
                                                  int64_t n) {
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (i >= n) return;
    const int64_t tg = i >> 2;
    const int row0 = (int)(tg / groups) * 16 + (int)(i & 3) * 4, g = (int)(tg % groups);
    unsigned w = 0;
    for (int j = 0; j < 4; ++j)
        if (row0 + j < N && g < have) w |= (zeros[(size_t)(row0 + j) * have + g] & 15u) << (4 * j);
    out[i] = (uint16_t)w;
}

// One group of one row per wave.
template <typename W, typename S>
__global__ void __launch_bounds__(64) k_q4_quantize(int K, int group, int have, const W *w, int64_t ldw,
                                                    uint8_t *codes, S *scales) {
    const int n = blockIdx.x / have, g = blockIdx.x - n * have, lane = threadIdx.x;
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
    if (lane == 0) scales[(size_t)n * have + g] = s;
}

struct Q4Args {
    const u32x4 *codes;
    const void *scales;
    const uint16_t *zeros;     // four outputs' zeros per value, or NULL
    const void *x;
    void *y;
    int64_t ldx, ldy;
    int N, K, kt, groups, rows;
};

// The bf16 terms of a value: TERMS = 1 for bf16, 2 for fp16, 3 for fp32.
template <typename V> struct Terms;
template <> struct Terms<bf16_t> { static constexpr int n = 1; };
template <> struct Terms<f16_t> { static constexpr int n = 2; };
template <> struct Terms<float> { static constexpr int n = 3; };

__device__ __forceinline__ float cut(float &rest) {     // the leading 8 significand bits; rest keeps the others
    const float hi = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    rest -= hi;
    return hi;
}

__device__ __forceinline__ bf16x8 weights(unsigned w) {
    union {
        unsigned u[4];
        bf16x8 v;
    } r;
    r.u[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    r.u[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    r.u[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    r.u[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    return r.v;
}

// A workgroup of four waves takes 16 outputs; the waves take every fourth
// 128-wide step, and their sums meet in LDS.  CT column tiles of 16.
template <typename V, typename S, int GROUP, int CT>
__global__ void __launch_bounds__(256) k_q4(Q4Args p) {
    constexpr int TERMS = Terms<V>::n;
    __shared__ float part[4][CT][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, kq = lane >> 4;
    const int64_t tile = blockIdx.x;
    f32x4 y[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int t = wave; t < p.kt; t += 4) {
        const u32x4 w = p.codes[(tile * p.kt + t) * 64 + lane];
        f32x4 acc[CT];
        float sum[CT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if ((s * 32) % GROUP == 0)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f}, sum[c] = 0.f;
            const bf16x8 a = weights(w[s]);
            const int k0 = t * 128 + s * 32 + kq * 8;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int xr = (c * 16 + col) / TERMS, term = (c * 16 + col) % TERMS;
                bf16x8 b;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = xr < p.rows && k0 + j < p.K
                                  ? (float)static_cast<const V *>(p.x)[xr * p.ldx + k0 + j] : 0.f;
                    float hi = v;
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) {
                        const float h = cut(v);
                        if (i == term) hi = h;
                    }
                    b[j] = (__bf16)hi;
                    sum[c] += hi;
                }
                acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc[c], 0, 0, 0);
            }
            if ((s + 1) * 32 % GROUP == 0) {
                const int g = (t * 128 + s * 32) / GROUP;
                const int64_t at = (tile * p.groups + g) * 16 + kq * 4;
                const unsigned z = p.zeros ? p.zeros[at >> 2] : 0x8888u;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    float x = sum[c];
                    x += __shfl_xor(x, 16, 64);
                    x += __shfl_xor(x, 32, 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float zero = (float)(16 + ((z >> (4 * i)) & 15u));
                        const float scale = (float)static_cast<const S *>(p.scales)[at + i];
                        y[c][i] = fmaf(scale, fmaf(-zero, x, acc[c][i]), y[c][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][c][kq * 4 + i][col] = y[c][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * p.rows; i += 256) {
        const int n = i & 15, r = i >> 4;
        float v = 0.f;
#pragma unroll
        for (int j = TERMS - 1; j >= 0; --j) {
            const int k = r * TERMS + j;
            float q = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) q += part[u][k >> 4][n][k & 15];
            v += q;
        }
        if (tile * 16 + n < p.N) static_cast<V *>(p.y)[r * p.ldy + tile * 16 + n] = (V)v;
    }
}

template <typename V, typename S, int GROUP>
void q4_launch(const Q4Args &a, hipStream_t st) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), wg(256);
    const int tiles = (a.rows * Terms<V>::n + 15) / 16;
    if (tiles == 1) hipLaunchKernelGGL((k_q4<V, S, GROUP, 1>), grid, wg, 0, st, a);
    if constexpr (Terms<V>::n > 1)
        if (tiles == 2) hipLaunchKernelGGL((k_q4<V, S, GROUP, 2>), grid, wg, 0, st, a);
    if constexpr (Terms<V>::n > 2)
        if (tiles == 3) hipLaunchKernelGGL((k_q4<V, S, GROUP, 3>), grid, wg, 0, st, a);
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

template <typename W>
void quantize(const fi_q4_desc *q, int have, const void *w, int64_t ldw, uint8_t *codes, void *scales,
              hipStream_t st) {
    const dim3 grid((unsigned)((size_t)q->N * have)), wg(64);
    if (q->scale_dtype == FI_F32)
        hipLaunchKernelGGL((k_q4_quantize<W, float>), grid, wg, 0, st, q->K, q->group, have, (const W *)w, ldw, codes,
                           (float *)scales);
    else if (q->scale_dtype == FI_BF16)
        hipLaunchKernelGGL((k_q4_quantize<W, bf16_t>), grid, wg, 0, st, q->K, q->group, have, (const W *)w, ldw,
                           codes, (bf16_t *)scales);
    else
        hipLaunchKernelGGL((k_q4_quantize<W, f16_t>), grid, wg, 0, st, q->K, q->group, have, (const W *)w, ldw, codes,
                           (f16_t *)scales);
}

unsigned blocks(int64_t n) { return (unsigned)((n + 255) / 256); }

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
    hipLaunchKernelGGL(k_q4_codes, dim3(blocks(words)), dim3(256), 0, st, desc->N, desc->K, l.kt, codes,
                       (unsigned *)(to + l.codes), words);
    if (desc->scale_dtype == FI_F32)
        hipLaunchKernelGGL((k_q4_scales<float>), dim3(blocks(sc)), dim3(256), 0, st, desc->N, have, l.groups,
                           (const float *)scales, (float *)(to + l.scales), sc);
    else    // both 16-bit types are copied as they are
        hipLaunchKernelGGL((k_q4_scales<bf16_t>), dim3(blocks(sc)), dim3(256), 0, st, desc->N, have, l.groups,
                           (const bf16_t *)scales, (bf16_t *)(to + l.scales), sc);
    if (zeros)
        hipLaunchKernelGGL(k_q4_zeros, dim3(blocks(sc / 4)), dim3(256), 0, st, desc->N, have, l.groups, zeros,
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
    if ((size_t)desc->N * have > 0x7fffffffu) return op_fail(FI_EINVAL, call, "too many groups");
    const size_t nk = (size_t)desc->N * desc->K, sb = (size_t)desc->N * have * value_bytes(desc->scale_dtype);
    const View out[] = {{codes, 1, nk, nk}, {scales, 1, sb, sb}};
    const size_t ws = value_bytes(w_dtype);
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
    const View out = {y, rows, desc->N * es, a.ldy * es};
    const View in[] = {{x, rows, desc->K * es, a.ldx * es}, {packed, 1, l.total, l.total}};
    if (outputs_meet(&out, 1, in, 2)) return op_fail(FI_EINVAL, call, "y shares memory with another argument");
    a.codes = (const u32x4 *)((const char *)packed + l.codes);
    a.scales = (const char *)packed + l.scales;
    a.zeros = desc->has_zeros ? (const uint16_t *)((const char *)packed + l.zeros) : nullptr;
    a.x = x, a.y = y, a.N = desc->N, a.K = desc->K, a.kt = l.kt, a.groups = l.groups, a.rows = rows;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FI_F32) q4_launch<float>(a, desc->group, desc->scale_dtype, st);
    else if (dtype == FI_BF16) q4_launch<bf16_t>(a, desc->group, desc->scale_dtype, st);
    else q4_launch<f16_t>(a, desc->group, desc->scale_dtype, st);
    return op_launched(call);
}

}  // extern "C"
