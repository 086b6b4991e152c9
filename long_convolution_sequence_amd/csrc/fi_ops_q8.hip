// Products in 8-bit integers (fi_q8_*): y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k] + bias[n].
// Both matrices lie in the order in which the matrix instruction
// v_mfma_i32_16x16x64_i8 takes them: a piece of 16 rows x 64 values along k is 1 KB,
// lane l's 16 bytes are the values 16 (l / 16) .. + 15 of row l % 16; the pieces of
// 16 rows follow each other along k.  So a wave reads a piece as 1 KB in a row, from
// memory into LDS and from LDS into registers, without bank conflicts.  Sums are
// whole numbers of 32 bits and exact: 128 * 128 * K < 2^31 for K < 2^17.
#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kQ8MaxK = 131071;        // 128 * 128 * K < 2^31
constexpr int64_t kQ8MaxRows = int64_t(1) << 24;
constexpr int64_t kQ8MaxOutputs = int64_t(1) << 38;
constexpr int kQ8Piece = 1024;         // bytes of 16 rows x 64 values

using i32x4 = int __attribute__((ext_vector_type(4)));

// Values along k as they are kept, zeros behind K: whole pairs of pieces.
__host__ __device__ inline int64_t q8_padded(int K) { return (K + 127) / 128 * 128; }
inline int64_t q8_code_bytes(int64_t rows, int K) { return (rows + 15) / 16 * 16 * q8_padded(K); }

// Where the 16 values from k on (a multiple of 16) of a row lie.
__device__ __forceinline__ size_t q8_at(int64_t row, int k, int64_t kp) {
    return (size_t)(row >> 4) * 16 * kp + (size_t)(k >> 6) * kQ8Piece + ((k >> 4) & 3) * 256 + (row & 15) * 16;
}

__device__ __forceinline__ void put16(int8_t *to, const int (&c)[16]) {
    i32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = (c[4 * j] & 255) | (c[4 * j + 1] & 255) << 8 | (c[4 * j + 2] & 255) << 16 | c[4 * j + 3] << 24;
    *reinterpret_cast<i32x4 *>(to) = v;
}

// Codes [rows][K] into order, 16 values a thread; the rows and values behind the
// matrix are zeros.  Scales follow the codes.
__global__ void __launch_bounds__(256) k_q8_pack(const int8_t *codes, const float *scales, int64_t rows, int K,
                                                 int8_t *packed, float *out) {
    const int64_t kp = q8_padded(K), units = kp / 16, total = (rows + 15) / 16 * 16 * units;
    for (int64_t u = blockIdx.x * (int64_t)256 + threadIdx.x; u < total; u += gridDim.x * (int64_t)256) {
        const int64_t row = u / units;
        const int k = (int)(u - row * units) * 16;
        int8_t *to = packed + q8_at(row, k, kp);
        if (row < rows && k + 16 <= K) {
            using Bytes __attribute__((aligned(1))) = i32x4;
            *reinterpret_cast<i32x4 *>(to) = *reinterpret_cast<const Bytes *>(codes + row * K + k);
        } else {
            int c[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i] = row < rows && k + i < K ? codes[row * K + k + i] : 0;
            put16(to, c);
        }
        if (k == 0 && row < rows) out[row] = scales[row];
    }
}

// A row's largest |x| as the bits of a float: NaN and infinity pass every number.
template <typename T>
__device__ __forceinline__ unsigned magnitude(T v) { return __float_as_uint((float)v) & 0x7fffffffu; }

// The scale of a row whose largest |x| has these bits.
__device__ __forceinline__ float q8_scale(unsigned top) {
    return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.f;
}

__device__ __forceinline__ int q8_code(float x, float scale) {
    // a scale of zero or NaN gives zeros; one below the normal numbers has lost
    // digits, so the quotient may pass 127
    const float c = scale > 0.f ? rintf(x / scale) : 0.f;
    return (int)fminf(fmaxf(c, -127.f), 127.f);
}

// Sixteen values of a row from k on, zeros behind K.
template <typename T>
__device__ __forceinline__ void values16(T (&v)[16], const T *row, int k, int K) {
    if (k + 16 <= K) {
        constexpr int CH = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 16; i += CH) {
            const Chunk<T, CH> c = *reinterpret_cast<const Chunk<T, CH> *>(row + k + i);
#pragma unroll
            for (int j = 0; j < CH; ++j) v[i + j] = c[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = k + i < K ? row[k + i] : (T)0.f;
    }
}

// Scales and codes of rows of values: WAVES waves a row, a lane 16 neighbouring values at
// a time; the first HELD of them stay in registers from the search for the largest to the
// codes, what is behind is read again.  16384 x 4096 bf16 48 us alone, 70 in turn with the
// product (4.2 and 2.9 TB/s).
template <typename T, int WAVES>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) k_q8_quantize(const T *x, int64_t ld, int64_t rows, int K,
                                                                           int8_t *packed, float *scales) {
    constexpr int HELD = sizeof(T) == 2 ? 4 : 2;
    __shared__ unsigned tops[WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t kp = q8_padded(K), padded = (rows + 15) / 16 * 16;
    const int64_t row = WAVES == 1 ? blockIdx.x * (int64_t)4 + wave : blockIdx.x;
    if (row >= padded) return;
    const int first = ((WAVES == 1 ? 0 : wave * 64) + lane) * 16;
    constexpr int step = WAVES * 64 * 16;
    const T *from = x + row * ld;
    T held[HELD][16];
    unsigned top = 0;
    if (row < rows) {
#pragma unroll
        for (int h = 0; h < HELD; ++h) values16(held[h], from, min(first + h * step, K), K);
#pragma unroll
        for (int h = 0; h < HELD; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, magnitude(held[h][i]));
        for (int k = first + HELD * step; k < K; k += step) {
            T v[16];
            values16(v, from, k, K);
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, magnitude(v[i]));
        }
    }
#pragma unroll
    for (int s = 32; s; s >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, s, 64));
    if (WAVES > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = max(top, tops[w]);
    }
    const float scale = q8_scale(top);
    if (first == 0 && row < rows) scales[row] = scale;
    const auto codes = [&](const T (&v)[16], int k) {
        int c[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = row < rows ? q8_code((float)v[i], scale) : 0;
        put16(packed + q8_at(row, k, kp), c);
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h)
        if (first + h * step < kp) codes(held[h], first + h * step);
    for (int k = first + HELD * step; k < kp; k += step) {
        T v[16];
        if (row < rows) values16(v, from, min(k, K), K);
        codes(v, k);
    }
}

struct Q8Args {
    const int8_t *a, *w;
    const float *sa, *sw, *bias;
    void *y;
    int64_t M, N, ldy, kp;
};

// What a wave's lanes wrote to LDS is read by its other lanes: an order for the compiler
// alone (the wave's accesses to LDS run in order), which must not follow from what it
// knows of one lane's addresses.
__device__ __forceinline__ void wave_exchanged() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Outputs [BM rows][BN columns] of a workgroup, WM x WN waves; a stage of 128 values
// along k of both sides in LDS while the next is on its way.  Workgroup i runs on XCD
// i % 8: each XCD takes a run of tiles in groups of eight rows of tiles, so that what
// its workgroups read at a time meets in its L2.  16384 x 8192 x 4096: 920000 cycles, for
// 57% of which the matrix units are busy, the rest is the barrier a stage with what it
// waits for; 450 us (2.4 POP/s) at the clock that the card comes to after forty such
// products in a row, up to 595 before.  The outputs' stores are 40 us of it; all of a
// stage's operands read ahead of its products took 582 us where it took 500.
template <typename T, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM *WN * 64) k_q8_product(Q8Args p) {
    constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;      // pieces of a wave
    constexpr int PIECES = (BM + BN) / 16 * 2, EACH = PIECES / (WM * WN);
    static_assert(PIECES % (WM * WN) == 0, "the waves bring equal shares");
    extern __shared__ __align__(16) int8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const unsigned tm = (unsigned)((p.M + BM - 1) / BM), tn = (unsigned)((p.N + BN - 1) / BN);
    const unsigned tile = blockIdx.x % 8 * ((tm * tn + 7) / 8) + blockIdx.x / 8;
    if (tile >= tm * tn || blockIdx.x / 8 >= (tm * tn + 7) / 8) return;
    const unsigned group = tile / (8 * tn), high = min(8u, tm - group * 8), at = tile - group * 8 * tn;
    const int64_t m0 = (group * 8 + at % high) * (int64_t)(BM / 16), n0 = at / high * (int64_t)(BN / 16);   // in pieces
    const int64_t mp = (p.M + 15) / 16, np = (p.N + 15) / 16;
    const int steps = (int)(p.kp / 128);

    const auto bring = [&](int step, int buffer) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int piece = wave * EACH + i, row = piece / 2;
            // rows behind the matrix: the last one again
            const int8_t *from;
            if (row < BM / 16)
                from = p.a + min(m0 + row, mp - 1) * 16 * p.kp;
            else
                from = p.w + min(n0 + row - BM / 16, np - 1) * 16 * p.kp;
            from += (size_t)step * (2 * kQ8Piece) + (piece & 1) * kQ8Piece + lane * 16;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                             (__attribute__((address_space(3))) void *)(lds + buffer * PIECES * kQ8Piece +
                                                                                        piece * kQ8Piece),
                                             16, 0, 0);
        }
    };

    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    bring(0, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) bring(s + 1, (s + 1) & 1);
        const int8_t *at = lds + (s & 1) * PIECES * kQ8Piece + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 fa[FM], fw[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[i] = *reinterpret_cast<const i32x4 *>(at + ((wm * FM + i) * 2 + h) * kQ8Piece);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fw[j] = *reinterpret_cast<const i32x4 *>(at + ((BM / 16 + wn * FN + j) * 2 + h) * kQ8Piece);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fa[i], acc[i][j], 0, 0, 0);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the next stage has arrived
        __syncthreads();
    }
    // Lane l holds outputs n = 4 (l / 16) .. + 3 of row m = l % 16: 16 rows at a time go
    // through a wave's own part of LDS, so that their stores are whole lines.
    T *y = static_cast<T *>(p.y);
    constexpr int W = FN * 16, PITCH = W + 16 / sizeof(T), CH = 16 / sizeof(T), LANES = W / CH;
    static_assert(WM * WN * 16 * PITCH * sizeof(T) <= 2 * PIECES * kQ8Piece, "the waves' parts fit");
    T *const mine = reinterpret_cast<T *>(lds) + wave * 16 * PITCH;
    const int64_t nw = (n0 + wn * FN) * 16;
    const bool whole = nw + W <= p.N;
    float sw[FN][4], bias[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t n = min(nw + j * 16 + (lane >> 4) * 4 + r, p.N - 1);
            sw[j][r] = p.sw[n];
            bias[j][r] = p.bias ? p.bias[n] : 0.f;
        }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t mw = (m0 + wm * FM + i) * 16;
        const float sa = p.sa[min(mw + (lane & 15), p.M - 1)];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mine[(lane & 15) * PITCH + j * 16 + (lane >> 4) * 4 + r] =
                    (T)fmaf((float)acc[i][j][r] * sa, sw[j][r], bias[j][r]);
        wave_exchanged();
        for (int u = lane; u < 16 * LANES; u += 64) {
            const int64_t m = mw + u / LANES, n = nw + u % LANES * CH;
            if (m >= p.M) continue;
            const Chunk<T, CH> v = *reinterpret_cast<const Chunk<T, CH> *>(mine + u / LANES * PITCH + u % LANES * CH);
            if (whole)
                *reinterpret_cast<Chunk<T, CH> *>(y + m * p.ldy + n) = v;
            else
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (n + e < p.N) y[m * p.ldy + n + e] = v[e];
        }
        wave_exchanged();
    }
}

// Up to 16 rows: 16 outputs a workgroup, its four waves share k.  HBM-bound: one row,
// 28672 x 8192, 36 us (6.6 TB/s: part of the weights stays in the last-level cache).
template <typename T>
__global__ void __launch_bounds__(256) k_q8_few(Q8Args p) {
    __shared__ i32x4 join[3][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int steps = (int)(p.kp / 64);
    const int row = min(lane & 15, (int)p.M - 1);             // of a: the rows behind it give outputs that are not kept
    const int8_t *a = p.a + (lane >> 4) * 256 + row * 16, *w = p.w + (size_t)blockIdx.x * 16 * p.kp + lane * 16;
    i32x4 acc{0, 0, 0, 0};
#pragma unroll 4
    for (int s = wave; s < steps; s += 4)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4 *>(w + (size_t)s * kQ8Piece),
                                                    *reinterpret_cast<const i32x4 *>(a + (size_t)s * kQ8Piece), acc, 0, 0,
                                                    0);
    if (wave) join[wave - 1][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 0; i < 3; ++i) acc += join[i][lane];
    const int64_t m = lane & 15, n = blockIdx.x * (int64_t)16 + (lane >> 4) * 4;
    if (m >= p.M) return;
    const float sa = p.sa[m];
    T *y = static_cast<T *>(p.y) + m * p.ldy;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (n + r < p.N) y[n + r] = (T)fmaf((float)acc[r] * sa, p.sw[n + r], p.bias ? p.bias[n + r] : 0.f);
}

template <typename T>
void launch_product(const Q8Args &p, hipStream_t st) {
    if (p.M <= 16) {
        hipLaunchKernelGGL((k_q8_few<T>), dim3((unsigned)((p.N + 15) / 16)), dim3(256), 0, st, p);
        return;
    }
    const auto tiles = [&](int64_t b) { return ((p.M + b - 1) / b) * ((p.N + b - 1) / b); };
    const auto run = [&](auto kernel, int64_t b, int waves) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((tiles(b) + 7) / 8 * 8)), dim3(waves * 64), 2 * (2 * b) / 16 * 2 * kQ8Piece, st, p);
    };
    // the largest tiles that still fill the card: 512 x 4096 x 4096 17 us with tiles of 64,
    // 27 with 128, 47 with 256; 1024 x 4096 x 4096 32, 31, 48; 8192 x 2592 x 864 42, 37, 39;
    // 16384 x 8192 x 4096 in tiles of 128 955 us, of 256 863 (before whole-line stores)
    if (tiles(256) >= 192) run(k_q8_product<T, 256, 256, 2, 4>, 256, 8);
    else if (tiles(128) >= 192) run(k_q8_product<T, 128, 128, 2, 2>, 128, 4);
    else run(k_q8_product<T, 64, 64, 2, 2>, 64, 4);
}

// Eight waves a row where one a row would leave the card idle: rows of 4096, 256 of them
// 6.7 us with eight and 6.8 with one, 1024 of them 13.3 and 7.6; 333 rows of 4999 8.9
// and 10.8.
template <typename T>
void quantize(const T *x, int64_t ld, int64_t rows, int K, int8_t *codes, float *scales, hipStream_t st) {
    const int64_t padded = (rows + 15) / 16 * 16;
    if (rows * 12 < K)
        hipLaunchKernelGGL((k_q8_quantize<T, 8>), dim3((unsigned)padded), dim3(512), 0, st, x, ld, rows, K, codes, scales);
    else
        hipLaunchKernelGGL((k_q8_quantize<T, 1>), dim3((unsigned)(padded / 4)), dim3(256), 0, st, x, ld, rows, K, codes, scales);
}

const char *q8_check(int64_t rows, int K) {
    if (rows < 0 || rows > kQ8MaxRows) return "rows is not in 0 .. 2^24";
    if (K < 1 || K > kQ8MaxK) return "K is not in 1 .. 131071";
    return nullptr;
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_q8_bytes(int64_t rows, int K) {
    if (q8_check(rows, K)) return 0;
    return up256((size_t)q8_code_bytes(rows, K)) + up256((size_t)rows * 4);
}

fi_status fi_q8_pack(int64_t rows, int K, const int8_t *codes, const float *scales, void *packed, void *stream) {
    static const char *call = "fi_q8_pack";
    if (const char *why = q8_check(rows, K)) return op_fail(FI_EINVAL, call, why);
    if (rows == 0) return FI_OK;
    if (!codes || !scales || !packed || (uintptr_t)packed % 256)
        return op_fail(FI_EINVAL, call, "codes, scales and packed memory aligned to 256 bytes are required");
    if (!aligned(4, {scales})) return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const size_t bytes = fi_q8_bytes(rows, K);
    const View out = {packed, 1, bytes, bytes};
    const View in[] = {{codes, 1, (size_t)rows * K, (size_t)rows * K}, {scales, 1, (size_t)rows * 4, (size_t)rows * 4}};
    if (outputs_meet(&out, 1, in, 2)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    const int64_t units = q8_code_bytes(rows, K) / 16;
    hipLaunchKernelGGL(k_q8_pack, dim3((unsigned)std::min<int64_t>((units + 255) / 256, 1 << 16)), dim3(256), 0,
                       (hipStream_t)stream, codes, scales, rows, K, (int8_t *)packed,
                       (float *)((char *)packed + up256((size_t)q8_code_bytes(rows, K))));
    return op_launched(call);
}

fi_status fi_q8_quantize(int64_t rows, int K, int dtype, const void *x, int64_t ld_x, void *packed, void *stream) {
    static const char *call = "fi_q8_quantize";
    if (const char *why = q8_check(rows, K)) return op_fail(FI_EINVAL, call, why);
    if (!value_type(dtype)) return op_fail(FI_EINVAL, call, "dtype is none of FI_F32, FI_BF16, FI_F16");
    if (ld_x != 0 && (ld_x < K || ld_x > (int64_t(1) << 40))) return op_fail(FI_EINVAL, call, "a row pitch is less than K");
    if (rows == 0) return FI_OK;
    if (!x || !packed || (uintptr_t)packed % 256)
        return op_fail(FI_EINVAL, call, "x and packed memory aligned to 256 bytes are required");
    const size_t es = value_bytes(dtype), bytes = fi_q8_bytes(rows, K);
    if (!aligned(es, {x})) return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const int64_t ld = pitch_or(ld_x, K);
    const View out = {packed, 1, bytes, bytes}, in = {x, rows, K * es, ld * es};
    if (outputs_meet(&out, 1, &in, 1)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    int8_t *codes = (int8_t *)packed;
    float *scales = (float *)((char *)packed + up256((size_t)q8_code_bytes(rows, K)));
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FI_F32) quantize((const float *)x, ld, rows, K, codes, scales, st);
    else if (dtype == FI_BF16) quantize((const bf16_t *)x, ld, rows, K, codes, scales, st);
    else quantize((const f16_t *)x, ld, rows, K, codes, scales, st);
    return op_launched(call);
}

fi_status fi_q8_product(int64_t rows, int64_t N, int K, const void *a, const void *w, const float *bias, int dtype,
                        void *y, int64_t ld_y, void *stream) {
    static const char *call = "fi_q8_product";
    if (const char *why = q8_check(rows, K)) return op_fail(FI_EINVAL, call, why);
    if (N < 1 || N > kQ8MaxRows) return op_fail(FI_EINVAL, call, "N is not in 1 .. 2^24");
    if (rows * N > int64_t(1) << 42) return op_fail(FI_EINVAL, call, "rows * N is over 2^42");
    // tiles of 256 x 256 at 512 threads: with those at the edges 2^22 + 2^17 + 1 of them at most, and a launch
    // has less than 2^32 threads
    if (rows * N > kQ8MaxOutputs) return op_fail(FI_EINVAL, call, "too large for a launch: rows * N is over 2^38");
    if (!value_type(dtype)) return op_fail(FI_EINVAL, call, "dtype is none of FI_F32, FI_BF16, FI_F16");
    if (ld_y != 0 && (ld_y < N || ld_y > (int64_t(1) << 40))) return op_fail(FI_EINVAL, call, "a row pitch is less than N");
    if (rows == 0) return FI_OK;
    if (!a || !w || !y || (uintptr_t)a % 256 || (uintptr_t)w % 256)
        return op_fail(FI_EINVAL, call, "a, w (aligned to 256 bytes) and y are required");
    const size_t es = value_bytes(dtype);
    if (!aligned(es, {y}) || !aligned(4, {bias})) return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const int64_t ld = pitch_or(ld_y, N);
    const size_t ba = fi_q8_bytes(rows, K), bw = fi_q8_bytes(N, K);
    const View out = {y, rows, (size_t)N * es, (size_t)ld * es};
    const View in[] = {{a, 1, ba, ba}, {w, 1, bw, bw}, {bias, 1, (size_t)N * 4, (size_t)N * 4}};
    if (outputs_meet(&out, 1, in, 3)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    Q8Args p = {};
    p.a = (const int8_t *)a, p.w = (const int8_t *)w, p.bias = bias, p.y = y;
    p.sa = (const float *)((const char *)a + up256((size_t)q8_code_bytes(rows, K)));
    p.sw = (const float *)((const char *)w + up256((size_t)q8_code_bytes(N, K)));
    p.M = rows, p.N = N, p.ldy = ld, p.kp = q8_padded(K);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FI_F32) launch_product<float>(p, st);
    else if (dtype == FI_BF16) launch_product<bf16_t>(p, st);
    else launch_product<f16_t>(p, st);
    return op_launched(call);
}

}  // extern "C"
