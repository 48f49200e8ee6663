// Rows of the norms in shared memory: how a team of threads holds one, and how it is brought there.
//
// In rows on 16-byte boundaries a thread holds vectors of eight columns (kBlockRow: a block takes a row,
// kWarpRow: a warp does). Rows that start anywhere (kAnyRow, a block per row) are copied from the 16-byte
// boundary before them, and column c belongs to thread c mod the block's threads: single loads and stores of
// a warp then lie side by side, and a block of an 8-bit checkpoint is what a warp holds at one place.
#pragma once

#include "norm.cuh"
#include "ptx.cuh"

namespace rlk {

enum RowMode { kBlockRow, kWarpRow, kAnyRow };

constexpr uint64_t kNormWaitNs = 1000000000ull;

template <bool BF16>
__device__ __forceinline__ V8 read_vec(const char *row, int vec) {
    if (BF16) return bf16_pairs(*reinterpret_cast<const uint4 *>(row + vec * 16));
    const uint4 *q = reinterpret_cast<const uint4 *>(row + vec * 32);
    return f32_pairs(q[0], q[1]);
}
template <bool BF16>
__device__ __forceinline__ float read_one(const char *row, int col) {
    if (BF16) return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(row + col * 2) << 16);
    return *reinterpret_cast<const float *>(row + col * 4);
}
__device__ __forceinline__ void store_one(const RowMat &m, int64_t at, float v) {
    if (m.bf16)
        static_cast<__nv_bfloat16 *>(m.p)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(m.p)[at] = v;
}

// Eight fp32 values of a thread that wrote them itself, in two planes of four, so that a warp's accesses of 16 bytes lie
// side by side (32 bytes apart they meet in the same banks two by two).
__device__ __forceinline__ void write_planes(float *base, int vec, int vecs, const V8 &a) {
    float v[kVec];
    floats_of(a, v);
    reinterpret_cast<float4 *>(base)[vec] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(base)[vecs + vec] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ V8 read_planes(const float *base, int vec, int vecs) {
    const uint4 *q = reinterpret_cast<const uint4 *>(base);
    return f32_pairs(q[vec], q[vecs + vec]);
}

// A thread's i-th eight columns. Only the last ones may be cut off by the row's end, or not there at all.
template <int MODE, int VPT>
struct Columns {
    int t, T, cols;
    bool has_last, cut;
    __device__ __forceinline__ Columns(int t, int T, int cols) : t(t), T(T), cols(cols) {
        const int vec = t + (VPT - 1) * T;
        has_last = MODE == kAnyRow || vec * kVec < cols;
        cut = MODE == kAnyRow || (vec + 1) * kVec > cols;
    }
    // Keeps the compiler from holding the addresses of single columns, dozens of them, in registers from row to row.
    __device__ __forceinline__ void next_row() {
        if (MODE == kAnyRow) asm volatile("" : "+r"(t), "+r"(T));
    }
    __device__ __forceinline__ bool none(int i) const { return i == VPT - 1 && !has_last; }
    __device__ __forceinline__ int vec(int i) const { return t + i * T; }
    __device__ __forceinline__ int col(int i, int j) const { return MODE == kAnyRow ? t + (i * kVec + j) * T : vec(i) * kVec + j; }
    // eight single values, 0 past the row's end
    template <typename Get>
    __device__ __forceinline__ V8 singles(int i, Get get) const {
        V8 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int a = col(i, 2 * k), b = col(i, 2 * k + 1);
            r.p[k] = pack2(i < VPT - 1 || a < cols ? get(a) : 0.f, i < VPT - 1 || b < cols ? get(b) : 0.f);
        }
        return r;
    }
    template <bool BF16>
    __device__ __forceinline__ V8 read(const char *row, int i) const {
        if (MODE == kAnyRow) return singles(i, [&](int c) { return read_one<BF16>(row, c); });
        return read_vec<BF16>(row, vec(i));
    }
    __device__ __forceinline__ V8 params(const void *p, int bf16, int fast, int i, float missing) const {
        if (!p) return singles(i, [&](int) { return missing; });
        if (MODE == kAnyRow) return singles(i, [&](int c) { return load_param(p, bf16, c); });
        float v[kVec];
        load_params(p, bf16, fast, vec(i) * kVec, cols, v);
        return pairs_of(v);
    }
    // 0 in the place of what lies past the row's end
    __device__ __forceinline__ V8 cut_off(const V8 &a, int i) const {
        if (MODE != kAnyRow) return clipped(a, vec(i) * kVec, cols);
        float v[kVec];
        floats_of(a, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (col(i, j) >= cols) v[j] = 0.f;
        return pairs_of(v);
    }
    // A row of which `plain` (its type is BF16's, rows on 16-byte boundaries) was found out once for all rows.
    template <bool BF16>
    __device__ __forceinline__ void store_plain(void *row, int fast, int i, const V8 &a) const {
        float v[kVec];
        floats_of(a, v);
        const int at = vec(i) * kVec, end = i == VPT - 1 && cut ? cols : at + kVec;
        if (BF16)
            store_vec(static_cast<__nv_bfloat16 *>(row), at, end, true, v);
        else if (fast == 2 && at + kVec <= end)
            store_vec32(static_cast<float *>(row), at, v);
        else
            store_vec(static_cast<float *>(row), at, end, true, v);
    }
    __device__ __forceinline__ void store(const RowMat &m, int64_t row, int i, const V8 &a) const {
        float v[kVec];
        floats_of(a, v);
        if (MODE != kAnyRow) {
            store_row(m, row, vec(i) * kVec, cols, v);
            return;
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (i < VPT - 1 || col(i, j) < cols) store_one(m, row * m.ld + col(i, j), v[j]);
    }
};

// The bytes that a row's copy starts before the row.
template <int MODE>
__device__ __forceinline__ int row_shift(const char *row) { return MODE == kAnyRow ? (int)(reinterpret_cast<uintptr_t>(row) & 15u) : 0; }
// The bytes of the whole 16-byte pieces of memory that hold a row.
__device__ __forceinline__ uint32_t window(const char *row, int bytes) { return (uint32_t)(((int)(reinterpret_cast<uintptr_t>(row) & 15u) + bytes + 15) & ~15); }

}  // namespace rlk
