// Shared by the operators of a recurrent block (scan, norms, 4-bit products):
// value types, argument checks and the calling thread's error message.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstdio>
#include <initializer_list>

#include "../../include/fi.h"

namespace fi {

using bf16_t = __bf16;
using f16_t = _Float16;

// ---- host side ---------------------------------------------------------------

char *op_error();                             // the calling thread's message, kOpErrorBytes long
constexpr size_t kOpErrorBytes = 160;

inline fi_status op_fail(fi_status s, const char *call, const char *what) {
    std::snprintf(op_error(), kOpErrorBytes, "%s: %s", call, what);
    return s;
}

inline fi_status op_launched(const char *call) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? FI_OK : op_fail(FI_EDEVICE, call, hipGetErrorString(e));
}

inline size_t value_bytes(int dtype) { return dtype == FI_F32 ? 4 : 2; }
inline bool value_type(int dtype) { return dtype >= FI_F32 && dtype <= FI_F16; }

// One tensor argument as `rows` rows of `width` bytes, `pitch` bytes apart.
struct View {
    const void *p;
    int64_t rows;
    size_t width, pitch;
};

// Whether two views may share a byte.  Rows of equal pitch are compared by
// their places within the pitch, so column slices of one tensor are separate;
// views of different pitch whose extents meet are taken to overlap.
inline bool views_meet(const View &a, const View &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
    using Wide = unsigned __int128;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const Wide ea = (Wide)pa + (Wide)(a.rows - 1) * a.pitch + a.width;
    const Wide eb = (Wide)pb + (Wide)(b.rows - 1) * b.pitch + b.width;
    if (ea <= pb || eb <= pa) return false;
    if (a.pitch != b.pitch) return true;
    const size_t delta = pb >= pa ? (pb - pa) % a.pitch : (a.pitch - (pa - pb) % a.pitch) % a.pitch;
    return !(delta >= a.width && delta + b.width <= a.pitch);
}

inline bool same_view(const View &a, const View &b) { return a.p == b.p && a.pitch == b.pitch; }

// Whether any output meets an input or another output (null views never do).
inline bool outputs_meet(const View *out, int nout, const View *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (views_meet(out[i], out[j])) return true;
        for (int j = 0; j < nin; ++j)
            if (views_meet(out[i], in[j])) return true;
    }
    return false;
}

// Whether every pointer (null ones too) is aligned to `bytes`.
inline bool aligned(size_t bytes, std::initializer_list<const void *> pointers) {
    for (const void *p : pointers)
        if ((uintptr_t)p % bytes) return false;
    return true;
}

inline int64_t pitch_or(int64_t ld, int64_t width) { return ld ? ld : width; }

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// ---- device side -------------------------------------------------------------

// CH values side by side.  The pitch and the start of a row are any number of
// elements, so a chunk is aligned to its element only; global loads and stores
// of 4 to 16 bytes need no more on this target.
template <typename T, int CH>
using Chunk __attribute__((aligned(sizeof(T)))) = T __attribute__((ext_vector_type(CH)));

// A lane's chunk of a row of D >= CH columns that would begin at column c: it is
// read from `at` = min(c, D - CH), so always whole and inside the row, without a
// branch (a lane-by-lane tail costs its wave a wait for memory at every tensor).
// The lane owns the elements from `skip` on; the others are a neighbour's.
template <int CH>
struct Place {
    unsigned at;
    int skip;
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(int c, int D) {
        const int a = c < D - CH ? c : D - CH;
        at = (unsigned)a;
        skip = c - a < CH ? c - a : CH;
        // kept as a value of its own: as a sum the compiler would carry it, and
        // with it every address, in 64 bits a lane
        asm("" : "+v"(at));
    }
};

// The address of a row's element as a row address for the whole wave and a
// 32-bit byte offset of the lane.
template <typename T>
__device__ __forceinline__ const T *in_row(const T *row, unsigned at) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + at * (unsigned)sizeof(T));
}
template <typename T>
__device__ __forceinline__ T *in_row(T *row, unsigned at) {
    return reinterpret_cast<T *>(reinterpret_cast<char *>(row) + at * (unsigned)sizeof(T));
}

// STREAM: read past the caches' usual keeping.
template <typename T, int CH, bool STREAM = false>
__device__ __forceinline__ Chunk<T, CH> load_chunk(const T *row, const Place<CH> &w) {
    const Chunk<T, CH> *p = reinterpret_cast<const Chunk<T, CH> *>(in_row(row, w.at));
    return STREAM ? __builtin_nontemporal_load(p) : *p;
}

// TAIL: a chunk may be owned in part (D is no multiple of CH).  Whole chunks are
// marked as streamed: what is still to be read keeps its place in the caches
// (rows of 131072 x 864: 312 -> 302 us; a reader right behind is no slower).
template <bool TAIL, typename T, int CH>
__device__ __forceinline__ void store_chunk(T *row, const Place<CH> &w, Chunk<T, CH> v) {
    if (w.skip == 0)
        __builtin_nontemporal_store(v, reinterpret_cast<Chunk<T, CH> *>(in_row(row, w.at)));
    else if (TAIL && w.skip < CH) {
        T *to = in_row(row, w.at);
#pragma unroll
        for (int i = 1; i < CH; ++i)
            if (i >= w.skip) to[i] = v[i];
    }
}

// Sum over the 64 lanes, in every lane: shifts within rows of 16 lanes, then
// across the rows, on the vector ALU's lane shifts (no LDS traffic).
__device__ __forceinline__ float lanes_sum(float v) {
#define FI_LANE_ADD(ctrl, rows) \
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false))
    FI_LANE_ADD(0x111, 0xf);   // from 1, 2, 4, 8 lanes below, in the row
    FI_LANE_ADD(0x112, 0xf);
    FI_LANE_ADD(0x114, 0xf);
    FI_LANE_ADD(0x118, 0xf);
    FI_LANE_ADD(0x142, 0xa);   // a row's last lane into the next row
    FI_LANE_ADD(0x143, 0xc);   // the lower half's last lane into the upper half
#undef FI_LANE_ADD
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace fi
