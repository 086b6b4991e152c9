// Rows held in registers by teams of waves: what the norms share.
#pragma once
#include "fi_ops.h"

namespace fi {

constexpr int kRowLane = 16;           // values of a row per lane at most

// Waves of a team (below) for a row of D values.
inline int team_waves(int D) { return (D + 64 * kRowLane - 1) / (64 * kRowLane); }

// A row is held in registers by a team: one wave up to 1024 values (four teams
// to a workgroup, no barrier), else a workgroup of as many waves as the row
// needs.  A lane holds NC chunks of CH neighbouring values, CH chosen so that
// the widest tensor of the row is read 16 bytes at a time; a team's waves take
// alternate stretches.  A team keeps its columns' weights (and, backwards,
// their column sums) in registers over all its rows.
template <int CH, int NC, bool MULTI>
struct Team {
    Place<CH> at[NC];      // this lane's chunks
    bool first;            // the lane of column 0
    int waves, wave, lane;
    int64_t row, rows_step;
    int turn;

    __device__ __forceinline__ Team(int D) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = blockDim.x >> 6;
        turn = 0;
        const int start = ((MULTI ? wave * 64 : 0) + lane) * CH, step = (MULTI ? waves : 1) * 64 * CH;
#pragma unroll
        for (int j = 0; j < NC; ++j) at[j] = Place<CH>(start + j * step, D);
        first = start == 0;
        row = MULTI ? blockIdx.x : blockIdx.x * (int64_t)waves + wave;
        rows_step = MULTI ? gridDim.x : gridDim.x * (int64_t)waves;
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
    // Two sums at once.
    __device__ __forceinline__ void sums(float &v, float &w, float (*slots)[2][16]) {
        v = lanes_sum(v), w = lanes_sum(w);
        if (!MULTI) return;
        if (lane == 0) slots[turn][0][wave] = v, slots[turn][1][wave] = w;
        __syncthreads();
        v = w = 0.f;
        for (int i = 0; i < waves; ++i) v += slots[turn][0][i], w += slots[turn][1][i];
        turn ^= 1;
    }
    // Three.
    __device__ __forceinline__ void sums(float &v, float &w, float &x, float (*slots)[3][16]) {
        v = lanes_sum(v), w = lanes_sum(w), x = lanes_sum(x);
        if (!MULTI) return;
        if (lane == 0) slots[turn][0][wave] = v, slots[turn][1][wave] = w, slots[turn][2][wave] = x;
        __syncthreads();
        v = w = x = 0.f;
        for (int i = 0; i < waves; ++i) v += slots[turn][0][i], w += slots[turn][1][i], x += slots[turn][2][i];
        turn ^= 1;
    }
};

// A row's values as they are loaded.  ALL: the tensor is there; else a null one
// reads as zeros.
template <bool ALL, bool STREAM, typename T, int CH, int NC>
struct Raw {
    Chunk<T, CH> v[NC];

    template <bool MULTI>
    __device__ __forceinline__ void load(const void *p, int64_t ld, int64_t row, const Team<CH, NC, MULTI> &t) {
        if (!ALL && !p) {
#pragma unroll
            for (int j = 0; j < NC; ++j) v[j] = (Chunk<T, CH>)(T)0.f;
            return;
        }
        const T *from = static_cast<const T *>(p) + row * ld;
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = load_chunk<T, CH, STREAM>(from, t.at[j]);
    }
    __device__ __forceinline__ void get(float (&f)[NC * CH]) const {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < CH; ++i) f[j * CH + i] = (float)v[j][i];
    }
};

template <bool TAIL, typename T, int CH, int NC, bool MULTI>
__device__ __forceinline__ void store_row(const float (&v)[NC * CH], void *p, int64_t ld,
                                          const Team<CH, NC, MULTI> &t) {
    T *to = static_cast<T *>(p) + t.row * ld;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        Chunk<T, CH> raw;
#pragma unroll
        for (int i = 0; i < CH; ++i) raw[i] = (T)v[j * CH + i];
        store_chunk<TAIL, T, CH>(to, t.at[j], raw);
    }
}

// Sum of the squares of what this lane owns.
template <bool TAIL, int CH, int NC, bool MULTI>
__device__ __forceinline__ float squares(const float (&v)[NC * CH], const Team<CH, NC, MULTI> &t) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const float x = TAIL && i < t.at[j].skip ? 0.f : v[j * CH + i];
            c = fmaf(x, x, c);
        }
        s += t.at[j].skip < CH ? c : 0.f;
    }
    return s;
}

// One column of the workgroups' column sums part [groups][2][D]: 64 columns a
// workgroup of sixteen waves, which take every sixteenth group and are added in
// their order.  A wave's loads do not wait for each other.  True in the lanes
// that hold column i's sum.
__device__ __forceinline__ bool column_sum(const float *part, int D, int groups, int i, float &sum) {
    __shared__ float join[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float s = 0.f;
    if (i < 2 * D) {
#pragma unroll 8
        for (int g = wave; g < groups; g += 16) s += part[(size_t)g * 2 * D + i];
    }
    join[wave][lane] = s;
    __syncthreads();
    if (wave || i >= 2 * D) return false;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += join[w][lane];
    sum = s;
    return true;
}

}  // namespace fi
