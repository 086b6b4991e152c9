// The gated linear recurrence and its gradients (fi_scan_*).
//
// With d_t = 1 - sigmoid(z_t) and b_t = e(d_t) x_t a position is the map
// s -> s - d_t s + b_t, affine in the state, and so is a run of positions:
// s -> A s + S.  The gradients are the same recurrence from the end:
// D_t = dy_t + c, c <- D_t - d_t D_t.
//
// Where the gate is open (z >= 0) the state is updated as s - d s, never as a s
// with a = 1 - d rounded to fp32: for decays near one (a memory of thousands of
// positions) the rounding of a alone is a relative error of 2^-25 / d in the
// memory's length.  Where it is shut (z < 0) the same rounding would be the whole
// of a (from z = -17 on 1 - d is 0, and with it every gradient through the gate):
// there a = e^z d, and the update is a s.  A position keeps the smaller of the two
// (see Decay).  It costs selects: a training pass over 32768 x 4 x 768 bf16 takes 368 us
// where 1 - d alone took 349, 131072 x 864 bf16 forwards 161 for 157.
//
// One pass over the data (k_scan_tile, k_scan_back).  A workgroup holds a tile
// of kTile positions x 64 columns in registers: a lane has kStep positions of
// four neighbouring columns (a "segment"), 16 lanes cover the tile's columns, the
// other lanes and the waves go on in time.  Every lane forms its segment's map;
// the first wave (one column a lane now) joins the segments' maps to the tile's
// map, publishes it, and finds the state before the tile from the tiles before:
// the nearest one that has published its end state, and the maps in between.
// Tiles are numbered by a counter as workgroups begin, all columns of a time
// before the next time: a tile only waits for tiles with lower numbers, which
// are running or done, so every wait ends.
//
// The join is the same chain of fmas whichever tile the state was found at
// (s <- A s + S, tile after tile), so results do not depend on timing.
//
// What bounds it: the memory's bytes where there are many columns.  Forward
// 32768 x 4 x 768 bf16 128 us at least and 138 in the mean (4.7 and 4.4 TB/s of the
// 5.0 that a copy reaches, x and gate read, y written, all once), 8192 x 8 x 768 fp32
// padded 86 us; 131072 x 864 bf16 161 us (4.2): rows of 1728 bytes begin in the
// middle of a 128-byte line every other time, and two tiles fetch it (1.39 times the
// bytes through the L2).  Backward, 32768 x 4 x 768 bf16, 246 us at least and 261 in
// the mean (4.1 and 3.9): the vector ALU, about 70 operations a value, some of
// them roots and exponentials.  Few columns: the chain of tiles (see kNear).  One
// time step after the other, four columns a lane, took 315 us where this took 85
// (padded), 514 for 158.
//
// A tile of 256 x 64: 128-byte pieces of 16-bit rows, two tiles of eight waves on a
// CU at 128 registers (backwards over fp32 values one, at up to 159).  128 columns
// took 186 us where this took 170, 256 columns 274; four waves 206, twelve 177,
// sixteen 200.  All waves looking back at 32 tiles together: 210.
#include <type_traits>

#include "fi_ops.h"

namespace fi {

namespace {

constexpr int kStep = 8;                        // positions of a lane
constexpr int kRow = 16;                        // lanes along a row
constexpr int kWaves = 8;                       // waves of a tile at most
constexpr int kTile = kWaves * 64 / kRow * kStep;   // positions of a tile
// Tiles looked back at together.  A step along the chain of tiles takes about 1 us
// (a state out to memory and in again), so few columns, with many times under way,
// want it long: kFar where there are no more than kNarrow column tiles, 128525 x 81
// fp32 86 -> 59 us, x 384 bf16 92 -> 77, x 512 (eight) 100 -> 96 but its fp32
// training pass 387 -> 407.  With many columns the words cost more than the steps
// (131072 x 864 bf16 166 -> 183 us; kNear = 4 178, 5 174).
constexpr int kNear = 6, kFar = 16;
constexpr int kNarrow = 7;
// Lengths up to this run one position after the other, a lane its columns: a single
// token is one short kernel (2.8 us at 8 x 864).  At T = 16 the tile takes 229 us
// and this 172 with 4096 x 2048 columns, 5.3 and 6.5 with 8 x 864; at T = 8 209 and 90.
constexpr int kSerial = 16;
constexpr int kPolls = 1 << 20;                 // looks at unfinished tiles before a wait gives up

struct ScanArgs {
    const void *x, *gate, *dy;
    void *y, *dx, *dgate;
    const float *bias, *state, *dfinal;
    float *final, *dstate;
    const int32_t *lengths;
    float *saved;              // [tiles][R] state after each tile
    unsigned long long *link;  // [tiles][R] a tile's map, then its end state (see Link)
    unsigned *ticket;          // tiles begun
    float *pbias;              // [tiles][R] partial sums of the bias gradient
    int64_t T;
    int64_t ldx, ldg, ldy, lddy, lddx, lddg;
    int B, D;
    int tiles;                 // along T
    int lanes_row;             // lanes that cover one row of D columns
    int lanes_all;             // and all B rows
    int col_tiles;
};

// A position's decay, to the last digits whichever way its gate lies.  `w` is what
// is kept of it: -d = -1 / (1 + e^z) where the gate is open (z >= 0, or NaN), a = e^z d
// where it is shut.  Its sign bit tells which (d = 0 is -0, a = 0 is +0).
struct Decay {
    float w, d;
    bool open;
    __device__ __forceinline__ Decay(float z) {
        const float ez = __builtin_amdgcn_exp2f(z * 1.44269504088896f);
        d = __builtin_amdgcn_rcpf(1.f + ez);
        open = !(z < 0.f);
        w = open ? -d : ez * d;
    }
    // of a position past its row's length: it leaves the state
    __device__ __forceinline__ void none() { d = 0.f, w = -0.f, open = true; }
};
__device__ __forceinline__ bool is_open(float w) { return (int)__float_as_uint(w) < 0; }

// (1 - d) s, as s - d s or a s; and one position, (1 - d) s + b.
__device__ __forceinline__ float decayed(bool open, float w, float s) { return fmaf(w, s, open ? s : 0.f); }
__device__ __forceinline__ float moved(bool open, float w, float s, float b) {
    return (open ? s : 0.f) + fmaf(w, s, b);
}

template <int IN>
__device__ __forceinline__ float input_factor(float d) {
    if (IN == FI_SCAN_PLAIN) return 1.f;
    if (IN == FI_SCAN_CONVEX) return d;
    return __builtin_amdgcn_sqrtf(d * (2.f - d));
}

// The same from what is kept: d (2 - d) as 2d - d^2 or 1 - a^2, d x as d x or x - a x.
__device__ __forceinline__ float energy(bool open, float w) { return fmaf(-w, w, open ? -2.f * w : 1.f); }
template <int IN>
__device__ __forceinline__ float input_of(bool open, float w, float x) {
    if (IN == FI_SCAN_PLAIN) return x;
    if (IN == FI_SCAN_CONVEX) return fmaf(-w, x, open ? 0.f : x);
    return __builtin_amdgcn_sqrtf(energy(open, w)) * x;
}

// The state behind one position, and ds/dz there: the decay's part a d s_{t-1},
// with a d = |w| - w^2 whichever w is, and the input factor's.  One reciprocal root
// of d (2 - d) gives the energy factor (also left in e) and its slope -a^2 d / e (at d = 0 it is a
// finite number, and both are 0).
template <int IN>
__device__ __forceinline__ float slope_and_move(float w, float x, float &s, float &e) {
    const bool open = is_open(w);
    const float ad = fmaf(-fabsf(w), fabsf(w), fabsf(w)), before = s;
    if (IN != FI_SCAN_ENERGY) {
        s = moved(open, w, s, input_of<IN>(open, w, x));
        return ad * (IN == FI_SCAN_PLAIN ? before : before - x);
    }
    const float sq = energy(open, w), inv = __builtin_amdgcn_rsqf(fmaxf(sq, 0x1p-126f));
    const float a = (open ? 1.f : 0.f) + w;
    e = sq * inv;
    s = moved(open, w, s, e * x);
    return fmaf(ad, before, -(a * inv * ad) * x);
}

// ---- what passes between tiles -------------------------------------------------
//
// One 64-bit word per tile and column, written and read whole (relaxed atomics
// of device scope: the value is its own flag): all ones = nothing yet; else
// {A, S}, the tile's map; then {kDone, state}, the state at the tile's end.

constexpr unsigned long long kNothing = ~0ull;
constexpr unsigned kDone = 0xfffffffeu;         // a NaN that no sum or product gives

__device__ __forceinline__ void link_put(unsigned long long *at, unsigned a, float s) {
    unsigned v = __float_as_uint(s);
    if (v == 0xffffffffu) v = 0x7fc00000u;      // a NaN's payload must not read as kNothing
    __hip_atomic_store(at, (unsigned long long)a << 32 | v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void link_put_map(unsigned long long *at, float A, float S) {
    unsigned a = __float_as_uint(A);
    if (a >= kDone) a = 0x7fc00000u;
    link_put(at, a, S);
}

__device__ __forceinline__ unsigned long long link_get(const unsigned long long *at) {
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool link_done(unsigned long long v) { return (unsigned)(v >> 32) == kDone; }

// The state at the end of the tile before, for one column r, from the WINDOW tiles
// before.  `row` is this tile's row of words, `step` the words between tiles
// (negative: the tiles come from the end), `have` the number of tiles before it
// (>= 1).
template <int WINDOW>
__device__ __forceinline__ bool link_look(const unsigned long long *row, unsigned r, int64_t step, int have, float &s) {
    unsigned long long v[WINDOW];
#pragma unroll
    for (int i = 0; i < WINDOW; ++i) v[i] = i < have ? link_get(in_row(row - (i + 1) * step, r)) : kNothing;
    // the nearest tile with its state, if every nearer one has its map
    int found = -1;
    bool open = true;
#pragma unroll
    for (int i = 0; i < WINDOW; ++i) {
        open = open && v[i] != kNothing;
        if (open && link_done(v[i])) {
            found = i;
            open = false;
        }
    }
    if (found < 0) return false;
#pragma unroll
    for (int i = WINDOW - 1; i >= 0; --i) {
        const float lo = __uint_as_float((unsigned)v[i]);
        if (i == found) s = lo;
        if (i < found) s = fmaf(__uint_as_float((unsigned)(v[i] >> 32)), s, lo);
    }
    return true;
}

// Looks until it is found.  A wait that gives up leaves NaN.
template <int WINDOW>
__device__ __forceinline__ float link_state(const unsigned long long *row, unsigned r, int64_t step, int have) {
    float s = __uint_as_float(0x7fc00000u);
    for (int polls = 0; polls < kPolls && !link_look<WINDOW>(row, r, step, have, s); ++polls)
        __builtin_amdgcn_s_sleep(1);
    return s;
}

__global__ void __launch_bounds__(256) k_scan_clear(unsigned long long *link, size_t n, unsigned *ticket) {
    for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n; i += gridDim.x * (size_t)256) link[i] = kNothing;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
}

// ---- a lane's part of a tile ------------------------------------------------------

template <int CH>
struct Lane {
    Place<CH> w;
    int b;             // batch row
    int64_t t0, last;  // first position; the row's last position (0 if it has none)
    int live, inside;  // of its kStep positions: before the row's length, before T

    // column group g of the tile's column tile, positions from t0 on
    __device__ __forceinline__ Lane(const ScanArgs &p, int g, int64_t t0_) {
        const int in = g < p.lanes_all ? g : p.lanes_all - 1;
        b = in / p.lanes_row;
        w = Place<CH>((in - b * p.lanes_row) * CH, p.D);
        if (in != g) w.skip = CH;
        t0 = t0_;
        int64_t len = p.T;
        if (p.lengths) {
            const int64_t n = p.lengths[b];
            len = n < 0 ? 0 : n < p.T ? n : p.T;
        }
        live = clip(len - t0);
        inside = clip(p.T - t0);
        last = len > 0 ? len - 1 : 0;
    }
    // whether every lane of the wave has all its positions
    __device__ __forceinline__ bool full() const { return __builtin_amdgcn_ballot_w64(live < kStep) == 0; }
    static __device__ __forceinline__ int clip(int64_t n) { return n < 0 ? 0 : n < kStep ? (int)n : kStep; }
};

// kStep rows of a lane.  FULL: all of them are live; else a row past the length
// reads the last one before it (row 0 of an empty sequence), unused.
template <bool FULL, typename V, int CH>
__device__ __forceinline__ void load_steps(Chunk<V, CH> (&v)[kStep], const void *p, int64_t ld, const ScanArgs &q,
                                           const Lane<CH> &l) {
    const int64_t step = ld * q.B;
    const V *row = static_cast<const V *>(p) + l.b * ld + l.w.at;
    const int64_t t0 = FULL ? l.t0 : l.t0 < l.last ? l.t0 : l.last;
    row += t0 * step;
    const int most = l.live - 1;
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
        const int64_t i = FULL ? k : k <= most ? k : most > 0 ? most : 0;
        v[k] = *reinterpret_cast<const Chunk<V, CH> *>(row + i * step);
    }
}

// kStep rows of a lane, up to T; zeros past the row's length.
template <bool FULL, typename V, int CH>
__device__ __forceinline__ void store_steps(const float (&v)[kStep][CH], void *p, int64_t ld, const ScanArgs &q,
                                            const Lane<CH> &l) {
    const int64_t step = ld * q.B;
    V *row = static_cast<V *>(p) + l.b * ld + l.t0 * step;
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
        if (!FULL && k >= l.inside) break;
        Chunk<V, CH> c;
#pragma unroll
        for (int e = 0; e < CH; ++e) c[e] = (V)(FULL || k < l.live ? v[k][e] : 0.f);
        store_chunk<true, V, CH>(row + k * step, l.w, c);
    }
}

// This workgroup's tile: along T (from either end), and along the columns.  One
// tile a workgroup: with several, a tile's first loads wait in order behind the
// stores of the one before (228 us where this takes 135).
struct Tile {
    int j, c;
    __device__ __forceinline__ Tile(const ScanArgs &p, int *slot) {
        int n = blockIdx.x;
        if (p.tiles > 1) {
            if (threadIdx.x == 0) *slot = (int)atomicAdd(p.ticket, 1u);
            __syncthreads();
            n = __builtin_amdgcn_readfirstlane(*slot);
        }
        j = n / p.col_tiles;
        c = n - j * p.col_tiles;
    }
};

// The other row of 16 lanes of a pair of rows, and the other half of a wave:
// `lo` and `hi` are the values of the earlier and the later one, in both.
__device__ __forceinline__ void rows_pair(float x, float &lo, float &hi) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
}
__device__ __forceinline__ void halves_pair(float x, float &lo, float &hi) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
}

// The tile's columns, one a lane: lane i has element i % CH of the lane group i / CH.
template <int CH>
struct Column {
    unsigned r;     // b * D + column
    bool own;
    __device__ __forceinline__ Column(const ScanArgs &p, int c) {
        const int i = threadIdx.x & 63;
        const Lane<CH> l(p, c * kRow + (i / CH) % kRow, 0);
        const int e = i % CH;
        own = i < kRow * CH && e >= l.w.skip;
        r = (unsigned)l.b * (unsigned)p.D + l.w.at + e;
        asm("" : "+v"(r));
    }
};

// A wave's values of its positions put aside in LDS, and taken back: kFar words a
// lane and the values together are more registers than two tiles a CU leave.
template <typename T, int CH>
using Parked = T __attribute__((ext_vector_type(CH)))[kStep][64];

template <typename T, int CH, typename Values>
__device__ __forceinline__ void park(Parked<T, CH> &to, const Values &v) {
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int e = 0; e < CH; ++e) to[k][threadIdx.x & 63][e] = v[k][e];
}
template <typename T, int CH, typename Values>
__device__ __forceinline__ void unpark(const Parked<T, CH> &from, Values &v) {
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int e = 0; e < CH; ++e) v[k][e] = from[k][threadIdx.x & 63][e];
}

template <typename V, int IN, int CH, bool FAR>
__global__ void __launch_bounds__(kWaves * 64, 4) k_scan_tile(ScanArgs p) {
    constexpr int COLS = kRow * CH;
    __shared__ float2 maps[kWaves][COLS];        // the waves' maps
    __shared__ float from[kWaves][COLS];         // states before the waves' positions
    __shared__ Parked<float, CH> parkA, parkS;   // FAR: the first wave's maps while it looks back
    __shared__ int slot;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int g = lane % kRow, row = lane / kRow;
    const int64_t R = (int64_t)p.B * p.D;
    const Tile tile(p, &slot);
    const int j = tile.j, jc = tile.c;
    const Lane<CH> l(p, jc * kRow + g, (int64_t)j * kTile + (wave * (64 / kRow) + row) * kStep);
    const Column<CH> c(p, jc);
    const bool full = l.full();
    float A[kStep][CH], S[kStep][CH];
    const auto segment = [&](auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        Chunk<V, CH> xg[kStep], xx[kStep];
        load_steps<FULL, V, CH>(xg, p.gate, p.ldg, p, l);
        load_steps<FULL, V, CH>(xx, p.x, p.ldx, p, l);
        Chunk<float, CH> bias = (Chunk<float, CH>)0.f;
        if (p.bias) bias = load_chunk<float, CH>(p.bias, l.w);
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                Decay q((float)xg[k][e] + bias[e]);
                float b = input_factor<IN>(q.d) * (float)xx[k][e];
                if (!FULL && k >= l.live) q.none(), b = 0.f;
                const float a0 = k ? A[k ? k - 1 : 0][e] : 1.f, s0 = k ? S[k ? k - 1 : 0][e] : 0.f;
                A[k][e] = decayed(q.open, q.w, a0);
                S[k][e] = moved(q.open, q.w, s0, b);
            }
    };
    if (full) segment(std::true_type());
    else segment(std::false_type());

    // the wave's map, and the map of what lies before this row of lanes
    float Ab[CH], Sb[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        float a0, a1, s0, s1, pa0, pa1, ps0, ps1;
        rows_pair(A[kStep - 1][e], a0, a1);
        rows_pair(S[kStep - 1][e], s0, s1);
        halves_pair(a0 * a1, pa0, pa1);
        halves_pair(fmaf(a1, s0, s1), ps0, ps1);
        if (lane < kRow) maps[wave][g * CH + e] = make_float2(pa0 * pa1, fmaf(pa1, ps0, ps1));
        const float ea = row & 1 ? a0 : 1.f, es = row & 1 ? s0 : 0.f;
        Ab[e] = row & 2 ? ea * pa0 : ea;
        Sb[e] = row & 2 ? fmaf(ea, ps0, es) : es;
    }
    __syncthreads();

    if (wave == 0) {
        if constexpr (FAR) {
            park<float, CH>(parkA, A);
            park<float, CH>(parkS, S);
        }
        if (c.own) {
            unsigned long long *row = p.link + j * R;
            float At = 1.f, St = 0.f, s = 0.f;
#pragma unroll 8
            for (int i = 0; i < waves; ++i) {
                const float2 m = maps[i][lane];
                St = fmaf(m.x, St, m.y);
                At *= m.x;
            }
            if (j > 0) {
                if (j + 1 < p.tiles) link_put_map(in_row(row, c.r), At, St);
                s = link_state<FAR ? kFar : kNear>(row, c.r, R, j);
            } else if (p.state) {
                s = *in_row(p.state, c.r);
            }
            const float end = fmaf(At, s, St);
            if (j + 1 < p.tiles) link_put(in_row(row, c.r), kDone, end);
            if (p.saved) *in_row(p.saved + j * R, c.r) = end;
            if (p.final && j + 1 == p.tiles) *in_row(p.final, c.r) = end;
#pragma unroll 8
            for (int i = 0; i < waves; ++i) {
                from[i][lane] = s;
                const float2 m = maps[i][lane];
                s = fmaf(m.x, s, m.y);
            }
        }
        if constexpr (FAR) {
            unpark<float, CH>(parkA, A);
            unpark<float, CH>(parkS, S);
        }
    }
    __syncthreads();

#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float b = fmaf(Ab[e], from[wave][g * CH + e], Sb[e]);
#pragma unroll
        for (int k = 0; k < kStep; ++k) S[k][e] = fmaf(A[k][e], b, S[k][e]);
    }
    if (full) store_steps<true, V, CH>(S, p.y, p.ldy, p, l);
    else store_steps<false, V, CH>(S, p.y, p.ldy, p, l);
}

// Makes the compiler forget what it knows of a lane's values, and so form what
// follows from them again where it is needed instead of keeping it in registers
// from phase to phase (x and its products as floats: 185 to 249 registers, one
// tile a CU).
template <typename V, int CH>
__device__ __forceinline__ void forget(Chunk<V, CH> (&v)[kStep]) {
    using Bits __attribute__((ext_vector_type(CH * sizeof(V) / 4 > 1 ? CH * sizeof(V) / 4 : 2))) = unsigned;
    if constexpr (CH * sizeof(V) >= 8) {
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            Bits b = __builtin_bit_cast(Bits, v[k]);
            asm("" : "+v"(b));
            v[k] = __builtin_bit_cast(Chunk<V, CH>, b);
        }
    }
}
template <int CH>
__device__ __forceinline__ void forget(float (&v)[kStep][CH]) {
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int e = 0; e < CH; ++e) asm("" : "+v"(v[k][e]));
}

// Backwards.  The states before the segments come from the saved state before
// the tile; the gradients' chain from the tiles after it.  Both kinds of maps
// are formed in one go (they share A).
template <typename V, int IN, int CH, bool FAR>
__global__ void __launch_bounds__(kWaves * 64, sizeof(V) == 2 ? 4 : 2) k_scan_back(ScanArgs p) {
    constexpr int COLS = kRow * CH;
    // the energy factors take the place of x, where they fit it and the last phase
    // need not form them again (7390 x 3 x 768 training 100 -> 96 us; in registers of
    // their own, with 16-bit values, they spill: 32768 x 4 x 768 bf16 368 -> 388)
    constexpr bool FACTORS = IN == FI_SCAN_ENERGY && sizeof(V) == 4;
    __shared__ float mul[kWaves][COLS];          // the waves' A; then their sums of dz
    __shared__ float fwd[kWaves][COLS];          // S; then the states before the waves' positions
    __shared__ float rev[kWaves][COLS];          // S from the end; then c behind the waves' positions
    __shared__ Chunk<float, CH> behind[2][kWaves * 64];   // the lanes' maps of what lies behind them in their wave
    __shared__ Parked<V, CH> parkx, parkdy;      // FAR: the first wave's values while it looks back
    __shared__ Parked<float, CH> parkw;
    __shared__ int slot;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int g = lane % kRow, row = lane / kRow;
    const int64_t R = (int64_t)p.B * p.D;
    const Tile tile(p, &slot);
    const int j = p.tiles - 1 - tile.j, jc = tile.c;
    const Lane<CH> l(p, jc * kRow + g, (int64_t)j * kTile + (wave * (64 / kRow) + row) * kStep);
    const Column<CH> c(p, jc);
    const bool full = l.full();
    const bool link = wave == 0 && c.own;
    float s = 0.f;
    if (link) s = j ? p.saved[(j - 1) * R + c.r] : p.state ? p.state[c.r] : 0.f;

    float w[kStep][CH];                          // decays; in the end dx
    // this lane's maps: s -> A s + S, and from the end c -> A c + Z, Z the sum of
    // dy_k times the decays up to k
    float A[CH], S[CH], Z[CH];
    Chunk<V, CH> xx[kStep], dy[kStep];
    const auto read = [&](auto whole) {
        constexpr bool FULL = decltype(whole)::value;
        Chunk<V, CH> xg[kStep];
        load_steps<FULL, V, CH>(xg, p.gate, p.ldg, p, l);
        load_steps<FULL, V, CH>(xx, p.x, p.ldx, p, l);
        load_steps<FULL, V, CH>(dy, p.dy, p.lddy, p, l);
        Chunk<float, CH> bias = (Chunk<float, CH>)0.f;
        if (p.bias) bias = load_chunk<float, CH>(p.bias, l.w);
#pragma unroll
        for (int k = 0; k < kStep; ++k)
            if (!FULL && k >= l.live) xx[k] = dy[k] = (Chunk<V, CH>)(V)0.f;
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            float a = 1.f, s = 0.f, z = 0.f;
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                Decay q((float)xg[k][e] + bias[e]);
                if (!FULL && k >= l.live) q.none();
                w[k][e] = q.w;
                a = decayed(q.open, q.w, a);
                s = moved(q.open, q.w, s, input_factor<IN>(q.d) * (float)xx[k][e]);
                z = fmaf(a, (float)dy[k][e], z);
            }
            A[e] = a, S[e] = s, Z[e] = z;
            __builtin_amdgcn_sched_barrier(0);   // column after column: interleaved, all four would not fit the registers
        }
    };
    if (full) read(std::true_type());
    else read(std::false_type());
    // maps of what lies before this row of lanes in its wave, and behind it
    float Ab[CH], Sb[CH];
    Chunk<float, CH> Az, Zz;
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        float a0, a1, s0, s1, z0, z1, pa0, pa1, ps0, ps1, pz0, pz1;
        rows_pair(A[e], a0, a1);
        rows_pair(S[e], s0, s1);
        rows_pair(Z[e], z0, z1);
        halves_pair(a0 * a1, pa0, pa1);
        halves_pair(fmaf(a1, s0, s1), ps0, ps1);
        halves_pair(fmaf(a0, z1, z0), pz0, pz1);
        if (lane < kRow) {
            mul[wave][g * CH + e] = pa0 * pa1;
            fwd[wave][g * CH + e] = fmaf(pa1, ps0, ps1);
            rev[wave][g * CH + e] = fmaf(pa0, pz1, pz0);
        }
        const float ea = row & 1 ? a0 : 1.f, es = row & 1 ? s0 : 0.f;
        Ab[e] = row & 2 ? ea * pa0 : ea;
        Sb[e] = row & 2 ? fmaf(ea, ps0, es) : es;
        const float ha = row & 1 ? 1.f : a1, hz = row & 1 ? 0.f : z1;
        Az[e] = row & 2 ? ha : ha * pa1;
        Zz[e] = row & 2 ? hz : fmaf(ha, pz1, hz);
    }
    behind[0][threadIdx.x] = Az;
    behind[1][threadIdx.x] = Zz;
    __syncthreads();

    float At = 1.f, Zt = 0.f;
    unsigned long long *links = p.link + j * R;
    if (link) {
#pragma unroll 8
        for (int i = waves - 1; i >= 0; --i) {
            Zt = fmaf(mul[i][lane], Zt, rev[i][lane]);
            At *= mul[i][lane];
        }
        if (j > 0 && j + 1 < p.tiles) link_put_map(in_row(links, c.r), At, Zt);
#pragma unroll 8
        for (int i = 0; i < waves; ++i) {
            const float S = fwd[i][lane];
            fwd[i][lane] = s;
            s = fmaf(mul[i][lane], s, S);
        }
    }
    __syncthreads();

    if (wave == 0) {
        if constexpr (FAR) {
            park<V, CH>(parkx, xx);
            park<V, CH>(parkdy, dy);
            park<float, CH>(parkw, w);
        }
        if (link) {
            float z = 0.f;
            if (j + 1 < p.tiles) z = link_state<FAR ? kFar : kNear>(links, c.r, -R, p.tiles - 1 - j);
            else if (p.dfinal) z = p.dfinal[c.r];
            const float end = fmaf(At, z, Zt);
            if (j > 0) link_put(in_row(links, c.r), kDone, end);
            else if (p.dstate) p.dstate[c.r] = end;
#pragma unroll 8
            for (int i = waves - 1; i >= 0; --i) {
                const float Z = rev[i][lane];
                rev[i][lane] = z;
                z = fmaf(mul[i][lane], z, Z);
            }
        }
        if constexpr (FAR) {
            unpark<V, CH>(parkx, xx);
            unpark<V, CH>(parkdy, dy);
            unpark<float, CH>(parkw, w);
        }
    }
    // ds/dz of every position (the other waves while the first one looks)
    forget(xx);
    forget(dy);
    forget(w);
    float slope[kStep][CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        float b = fmaf(Ab[e], fwd[wave][g * CH + e], Sb[e]);
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float factor = 0.f;
            slope[k][e] = slope_and_move<IN>(w[k][e], (float)xx[k][e], b, factor);
            if constexpr (FACTORS) xx[k][e] = factor;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();

    forget(w);
    Az = behind[0][threadIdx.x];
    Zz = behind[1][threadIdx.x];
    float sum[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        float b = fmaf(Az[e], rev[wave][g * CH + e], Zz[e]);
        sum[e] = 0.f;
#pragma unroll
        for (int k = kStep - 1; k >= 0; --k) {
            const float G = (float)dy[k][e] + b;
            const bool open = is_open(w[k][e]);
            b = decayed(open, w[k][e], G);
            slope[k][e] *= G;
            sum[e] += slope[k][e];     // 0 past the row's length: d = x = 0 there
            w[k][e] = FACTORS ? (float)xx[k][e] * G : input_of<IN>(open, w[k][e], G);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if (full) {
        store_steps<true, V, CH>(w, p.dx, p.lddx, p, l);
        store_steps<true, V, CH>(slope, p.dgate, p.lddg, p, l);
    } else {
        store_steps<false, V, CH>(w, p.dx, p.lddx, p, l);
        store_steps<false, V, CH>(slope, p.dgate, p.lddg, p, l);
    }
    if (p.pbias) {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            float s0, s1;
            rows_pair(sum[e], s0, s1);
            halves_pair(s0 + s1, s0, s1);
            if (lane < kRow) mul[wave][g * CH + e] = s0 + s1;
        }
        __syncthreads();
        if (link) {
            float t = 0.f;
#pragma unroll 8
            for (int i = 0; i < waves; ++i) t += mul[i][lane];
            p.pbias[j * R + c.r] = t;
        }
    }
}

// Short lengths: a lane runs its columns from the first position to the last,
// reading ahead; nothing passes between lanes.
template <typename V, int IN, int CH>
__global__ void __launch_bounds__(64) k_scan_serial(ScanArgs p) {
    const int g = blockIdx.x * 64 + threadIdx.x;
    if (g >= p.lanes_all) return;
    const Lane<CH> l(p, g, 0);
    int64_t len = p.T;
    if (p.lengths) {
        const int64_t n = p.lengths[l.b];
        len = n < 0 ? 0 : n < p.T ? n : p.T;
    }
    const size_t r = (size_t)l.b * p.D;
    const V *gate = static_cast<const V *>(p.gate) + l.b * p.ldg + l.w.at;
    const V *x = static_cast<const V *>(p.x) + l.b * p.ldx + l.w.at;
    V *y = static_cast<V *>(p.y) + l.b * p.ldy;
    Chunk<float, CH> bias = (Chunk<float, CH>)0.f, s = (Chunk<float, CH>)0.f;
    Chunk<V, CH> ng = *reinterpret_cast<const Chunk<V, CH> *>(gate), nx = *reinterpret_cast<const Chunk<V, CH> *>(x);
    if (p.bias) bias = load_chunk<float, CH>(p.bias, l.w);
    if (p.state) s = load_chunk<float, CH>(p.state + r, l.w);
    for (int64_t t = 0; t < p.T; ++t) {
        const Chunk<V, CH> cg = ng, cx = nx;
        if (t + 1 < p.T) {
            ng = *reinterpret_cast<const Chunk<V, CH> *>(gate + (t + 1) * p.B * p.ldg);
            nx = *reinterpret_cast<const Chunk<V, CH> *>(x + (t + 1) * p.B * p.ldx);
        }
        Chunk<V, CH> out = (Chunk<V, CH>)(V)0.f;
        if (t < len) {
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                const Decay q((float)cg[e] + bias[e]);
                s[e] = moved(q.open, q.w, s[e], input_factor<IN>(q.d) * (float)cx[e]);
                out[e] = (V)s[e];
            }
        }
        store_chunk<true, V, CH>(y + t * p.B * p.ldy, l.w, out);
    }
    if (p.saved) store_chunk<true, float, CH>(p.saved + r, l.w, s);
    if (p.final) store_chunk<true, float, CH>(p.final + r, l.w, s);
}

// dbias: the tiles' and rows' partial sums of 64 channels a workgroup; its
// sixteen waves take every sixteenth row and are added in their order.
__global__ void __launch_bounds__(1024) k_scan_dbias(ScanArgs p, float *dbias) {
    __shared__ float join[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < p.D) {
#pragma unroll 8
        for (int64_t i = wave; i < (int64_t)p.tiles * p.B; i += 16) s += p.pbias[i * p.D + c];
    }
    join[wave][lane] = s;
    __syncthreads();
    if (wave || c >= p.D) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += join[w][lane];
    dbias[c] = s;
}

// T = 0: the state passes through.
__global__ void __launch_bounds__(64) k_scan_pass(const float *from, float *to, size_t n) {
    const size_t i = blockIdx.x * (size_t)64 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.f;
}

struct Plan {
    size_t R;
    int64_t tiles;
    size_t part;       // bytes of one fp32 [tiles][R] array
    size_t link;       // bytes of the words between tiles and their counter, 0 for one tile
};

const char *scan_plan(const fi_scan_desc *q, Plan &p) {
    if (!q) return "null descriptor";
    if (q->T < 0 || q->batch < 1 || q->channels < 1) return "T >= 0, batch >= 1 and channels >= 1 are needed";
    if (!value_type(q->dtype)) return "dtype is none of FI_F32, FI_BF16, FI_F16";
    if (q->input < FI_SCAN_PLAIN || q->input > FI_SCAN_ENERGY) return "input is none of FI_SCAN_*";
    const int64_t ld[] = {q->ld_x, q->ld_gate, q->ld_y, q->ld_dy, q->ld_dx, q->ld_dgate};
    for (int64_t v : ld)
        if (v != 0 && (v < q->channels || v > (int64_t(1) << 40))) return "a row pitch is less than channels";
    for (int v : q->reserved)
        if (v) return "reserved is not zero";
    p.R = (size_t)q->batch * q->channels;
    if (p.R > (size_t(1) << 24)) return "batch * channels is over 2^24";
    if (q->T > (int64_t(1) << 23)) return "T is over 2^23";
    p.tiles = (q->T + kTile - 1) / kTile;
    p.part = up256((size_t)p.tiles * p.R * sizeof(float));
    p.link = p.tiles > 1 ? up256((size_t)p.tiles * p.R * sizeof(unsigned long long)) + 256 : 0;
    // a launch has less than 2^32 threads, so less than 2^23 workgroups of 512; a
    // workgroup has 64 columns (no less than 40: rows of 5 are two groups of 4), or
    // 16 where rows have less than 4
    if (p.tiles * (int64_t)p.R > (int64_t(1) << (q->channels < 4 ? 26 : 28)))
        return "batch * channels * T is too large";
    return nullptr;
}

size_t scan_workspace(const Plan &p, bool backward) {
    return std::max<size_t>(p.link + (backward ? p.part : 0), 256);
}

// The counter, then the words between tiles (a backward pass keeps its sums behind them).
void scan_links(const Plan &pl, void *workspace, ScanArgs &a) {
    if (!pl.link) return;
    a.ticket = (unsigned *)workspace;
    a.link = (unsigned long long *)((char *)workspace + 256);
}

void scan_args(const fi_scan_desc *q, const Plan &pl, ScanArgs &a) {
    a.T = q->T;
    a.B = q->batch;
    a.D = q->channels;
    a.tiles = (int)pl.tiles;
    a.ldx = pitch_or(q->ld_x, a.D);
    a.ldg = pitch_or(q->ld_gate, a.D);
    a.ldy = pitch_or(q->ld_y, a.D);
    a.lddy = pitch_or(q->ld_dy, a.D);
    a.lddx = pitch_or(q->ld_dx, a.D);
    a.lddg = pitch_or(q->ld_dgate, a.D);
}

template <typename V, int IN, int CH>
void scan_launch(ScanArgs a, bool backward, hipStream_t st) {
    a.lanes_row = (a.D + CH - 1) / CH;
    a.lanes_all = a.lanes_row * a.B;
    a.col_tiles = (a.lanes_all + kRow - 1) / kRow;
    if (!backward && a.T <= kSerial) {
        hipLaunchKernelGGL((k_scan_serial<V, IN, CH>), dim3((a.lanes_all + 63) / 64), dim3(64), 0, st, a);
        return;
    }
    const unsigned per_wave = 64 / kRow * kStep;
    const unsigned waves = a.tiles > 1 ? kWaves : (unsigned)((a.T + per_wave - 1) / per_wave);
    if (a.tiles > 1) {
        const size_t n = (size_t)a.tiles * a.B * a.D;
        hipLaunchKernelGGL(k_scan_clear, dim3((unsigned)std::min<size_t>((n + 1023) / 1024, 4096)), dim3(256), 0, st,
                           a.link, n, a.ticket);
    }
    const dim3 grid((unsigned)a.tiles * a.col_tiles), wg(waves * 64);
    if (a.tiles > 1 && a.col_tiles <= kNarrow) {
        if (backward) hipLaunchKernelGGL((k_scan_back<V, IN, CH, true>), grid, wg, 0, st, a);
        else hipLaunchKernelGGL((k_scan_tile<V, IN, CH, true>), grid, wg, 0, st, a);
    } else if (backward) {
        hipLaunchKernelGGL((k_scan_back<V, IN, CH, false>), grid, wg, 0, st, a);
    } else {
        hipLaunchKernelGGL((k_scan_tile<V, IN, CH, false>), grid, wg, 0, st, a);
    }
}

// Lanes take four neighbouring columns, or one where a row has fewer.
template <typename V, int IN>
void scan_forward(const ScanArgs &a, hipStream_t st) {
    if (a.D < 4) scan_launch<V, IN, 1>(a, false, st);
    else scan_launch<V, IN, 4>(a, false, st);
}

template <typename V, int IN>
void scan_backward(const ScanArgs &a, hipStream_t st) {
    if (a.D < 4) scan_launch<V, IN, 1>(a, true, st);
    else scan_launch<V, IN, 4>(a, true, st);
}

using ScanLaunch = void (*)(const ScanArgs &, hipStream_t);

template <typename V>
ScanLaunch pick(int input, bool backward) {
    switch (input) {
        case FI_SCAN_PLAIN: return backward ? &scan_backward<V, FI_SCAN_PLAIN> : &scan_forward<V, FI_SCAN_PLAIN>;
        case FI_SCAN_CONVEX: return backward ? &scan_backward<V, FI_SCAN_CONVEX> : &scan_forward<V, FI_SCAN_CONVEX>;
        default: return backward ? &scan_backward<V, FI_SCAN_ENERGY> : &scan_forward<V, FI_SCAN_ENERGY>;
    }
}

ScanLaunch pick(int dtype, int input, bool backward) {
    return dtype == FI_F32 ? pick<float>(input, backward)
                           : dtype == FI_BF16 ? pick<bf16_t>(input, backward) : pick<f16_t>(input, backward);
}

}  // namespace

}  // namespace fi

using namespace fi;

extern "C" {

size_t fi_scan_saved_bytes(const fi_scan_desc *desc) {
    Plan pl;
    return scan_plan(desc, pl) ? 0 : std::max<size_t>(pl.part, 256);
}

size_t fi_scan_workspace_bytes(const fi_scan_desc *desc, int backward) {
    Plan pl;
    if (scan_plan(desc, pl)) return 0;
    return scan_workspace(pl, backward);
}

fi_status fi_scan_forward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                          const float *state, const int32_t *lengths, void *y, float *final, void *saved,
                          void *workspace, void *stream) {
    static const char *call = "fi_scan_forward";
    Plan pl;
    if (const char *why = scan_plan(desc, pl)) return op_fail(FI_EINVAL, call, why);
    const hipStream_t st = (hipStream_t)stream;
    ScanArgs a = {};
    scan_args(desc, pl, a);
    const size_t es = value_bytes(desc->dtype), w = a.D * es, fr = pl.R * sizeof(float);
    const int64_t rows = desc->T * a.B;
    const size_t ws = scan_workspace(pl, false);
    if (rows > 0 && (!x || !gate || !y || (!workspace && ws > 256)))
        return op_fail(FI_EINVAL, call, "x, gate, y and workspace are required");
    if ((uintptr_t)workspace % 256 || (uintptr_t)saved % 256)
        return op_fail(FI_EINVAL, call, "workspace and saved need an alignment of 256 bytes");
    if (!aligned(es, {x, gate, y}) || !aligned(4, {bias, state, lengths, final}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const View out[] = {{y, rows, w, a.ldy * es}, {final, 1, fr, fr}, {saved, 1, pl.part, pl.part},
                        {workspace, 1, ws, ws}};
    const View in[] = {{x, rows, w, a.ldx * es}, {gate, rows, w, a.ldg * es}, {bias, 1, a.D * 4u, a.D * 4u},
                       {lengths, 1, a.B * 4u, a.B * 4u}, {final == state ? nullptr : state, 1, fr, fr}};
    if (outputs_meet(out, 4, in, 5) || (final == state && views_meet({state, 1, fr, fr}, out[0])))
        return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    a.x = x, a.gate = gate, a.bias = bias, a.state = state, a.lengths = lengths;
    a.y = y, a.final = final, a.saved = (float *)saved;
    if (rows == 0) {
        if (final && final != state)
            hipLaunchKernelGGL(k_scan_pass, dim3((unsigned)((pl.R + 63) / 64)), dim3(64), 0, st, state, final, pl.R);
        return op_launched(call);
    }
    scan_links(pl, workspace, a);
    pick(desc->dtype, desc->input, false)(a, st);
    return op_launched(call);
}

fi_status fi_scan_backward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                           const float *state, const int32_t *lengths, const void *saved, const void *dy,
                           const float *dfinal, void *dx, void *dgate, float *dbias, float *dstate,
                           void *workspace, void *stream) {
    static const char *call = "fi_scan_backward";
    Plan pl;
    if (const char *why = scan_plan(desc, pl)) return op_fail(FI_EINVAL, call, why);
    const hipStream_t st = (hipStream_t)stream;
    ScanArgs a = {};
    scan_args(desc, pl, a);
    const size_t es = value_bytes(desc->dtype), w = a.D * es, fr = pl.R * sizeof(float);
    const int64_t rows = desc->T * a.B;
    if (rows > 0 && (!x || !gate || !saved || !dy || !dx || !dgate || !workspace))
        return op_fail(FI_EINVAL, call, "x, gate, saved, dy, dx, dgate and workspace are required");
    if ((uintptr_t)workspace % 256 || (uintptr_t)saved % 256)
        return op_fail(FI_EINVAL, call, "workspace and saved need an alignment of 256 bytes");
    if (!aligned(es, {x, gate, dy, dx, dgate}) || !aligned(4, {bias, state, lengths, dfinal, dbias, dstate}))
        return op_fail(FI_EINVAL, call, "a pointer is not aligned to its values");
    const size_t ws = scan_workspace(pl, true);
    const View out[] = {{dx, rows, w, a.lddx * es}, {dgate, rows, w, a.lddg * es}, {dbias, 1, a.D * 4u, a.D * 4u},
                        {dstate, 1, fr, fr}, {workspace, 1, ws, ws}};
    const View in[] = {{x, rows, w, a.ldx * es}, {gate, rows, w, a.ldg * es}, {dy, rows, w, a.lddy * es},
                       {bias, 1, a.D * 4u, a.D * 4u}, {lengths, 1, a.B * 4u, a.B * 4u}, {state, 1, fr, fr},
                       {dfinal, 1, fr, fr}, {saved, 1, pl.part, pl.part}};
    if (outputs_meet(out, 5, in, 8)) return op_fail(FI_EINVAL, call, "an output shares memory with another argument");
    a.x = x, a.gate = gate, a.bias = bias, a.state = state, a.lengths = lengths;
    a.saved = (float *)saved, a.dy = dy, a.dfinal = dfinal, a.dx = dx, a.dgate = dgate, a.dstate = dstate;
    const unsigned cols = (unsigned)((pl.R + 63) / 64);
    if (rows == 0) {
        if (dstate) hipLaunchKernelGGL(k_scan_pass, dim3(cols), dim3(64), 0, st, dfinal, dstate, pl.R);
    } else {
        scan_links(pl, workspace, a);
        // one tile of one row: its sums are the gradient
        const bool alone = pl.tiles == 1 && a.B == 1;
        a.pbias = dbias ? alone ? dbias : (float *)((char *)workspace + pl.link) : nullptr;
        pick(desc->dtype, desc->input, true)(a, st);
        if (alone) return op_launched(call);
    }
    if (dbias) hipLaunchKernelGGL(k_scan_dbias, dim3((unsigned)((a.D + 63) / 64)), dim3(1024), 0, st, a, dbias);
    return op_launched(call);
}

}  // extern "C"
