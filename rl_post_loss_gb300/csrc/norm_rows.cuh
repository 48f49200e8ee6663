// Rows of the norms in shared memory: how a team of threads holds one, and how it is brought there.
//
// In rows on 16-byte boundaries a thread holds vectors of eight columns (kBlockRow: a block takes a row, kWarpRow: a
// warp does). Rows that start anywhere are copied from the 16-byte boundary before them, and then a block per row goes one of two ways.
//   kShiftRow  Vectors again: a thread reads the 16-byte pieces that its vector lies in and shifts them into place, by whole
//              words first. Written, a warp's vectors are shifted the other way, with what each lane gets from the
//              one before it, so that stores are whole pieces of memory; a column that shares a piece with another warp's
//              columns is stored by itself.
//   kAnyRow    Column c belongs to thread c mod the block's threads, so that single loads and stores of a warp lie side by side.
// Shifting costs some 60 instructions a vector written, single columns cost an access each and 8-bit codes an encoding
// each. The backward pass shifts what it reads from codes (16000 x 3001 bf16 from int8: 124 us, single columns 154) and takes
// single columns else (8192 x 6145 bf16 layer norm 139 us, shifted 134; 8191 x 2050 fp32 51 and 60, 4000 x 15001 bf16 174 and 205).
#pragma once

#include "norm.cuh"
#include "ptx.cuh"

namespace rlk {

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

// Words from the by-th on, if `on`.
template <int COUNT, int BY, int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N], bool on) {
    static_assert(COUNT + BY <= N, "");
#pragma unroll
    for (int i = 0; i < COUNT; ++i) w[i] = on ? w[i + BY] : w[i];
}
__device__ __forceinline__ void put(uint32_t *w, uint4 a) { w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w; }

// Vector `vec` of a row that starts `shift` bytes into the pieces at `row`.
template <bool BF16>
__device__ __forceinline__ V8 read_shifted(const char *row, int shift, int vec) {
    constexpr int kPieces = BF16 ? 2 : 3;
    const uint4 *q = reinterpret_cast<const uint4 *>(row) + vec * (kPieces - 1);
    uint32_t w[4 * kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) put(w + 4 * k, q[k]);
    if constexpr (BF16) {
        shift_words<6, 2>(w, shift & 8);
        shift_words<5, 1>(w, shift & 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], shift * 8 & 16);
        return bf16_pairs(make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        shift_words<9, 2>(w, shift & 8);
        shift_words<8, 1>(w, shift & 4);
        return f32_pairs(make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
    }
}
// The same of a row of codes.
__device__ __forceinline__ uint2 codes_shifted(const char *row, int shift, int vec) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(row + (shift & ~3)) + vec * 2;
    const int by = (shift & 3) * 8;
    return make_uint2(__funnelshift_r(q[0], q[1], by), __funnelshift_r(q[1], q[2], by));
}

// Vector `vec` of a row of `cols` columns, by lanes that hold neighbouring vectors (`mask`: those lanes, from lane 0 on).
template <typename T, int N>
__device__ __forceinline__ void store_words(T *row, int vec, int cols, uint32_t mask, const uint32_t (&u)[N]) {
    constexpr bool kHalf = N == 4;           // two columns a word
    constexpr int kPiece = kHalf ? 8 : 4;    // columns
    constexpr int kBefore = kHalf ? 4 : 3;   // words of the lane before that may be needed
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T), col = vec * kVec, lane = threadIdx.x & 31;
    row += col;
    uint32_t w[kBefore + N];
#pragma unroll
    for (int k = 0; k < kBefore; ++k) w[k] = __shfl_up_sync(mask, u[N - kBefore + k], 1);
#pragma unroll
    for (int k = 0; k < N; ++k) w[kBefore + k] = u[k];
    // the piece that ends (fp32: the first one that does) among this lane's columns is whole, and so is that of the lane behind
    const bool mine = (lane > 0 || off == 0) && col - off + kVec <= cols;
    if constexpr (kHalf) {
        shift_words<4, 4>(w, off == 0);
        shift_words<6, 2>(w, (8 - off) & 4);
        shift_words<5, 1>(w, (8 - off) & 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], (off & 1) * 16);
        if (mine) *reinterpret_cast<uint4 *>(row - off) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        shift_words<9, 2>(w, (3 - off) & 2);
        shift_words<8, 1>(w, (3 - off) & 1);
        if (mine) *reinterpret_cast<uint4 *>(row - off) = make_uint4(w[0], w[1], w[2], w[3]);
        if (col - off + kVec <= cols) *reinterpret_cast<uint4 *>(row - off + kPiece) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    if (col + (32 - lane) * kVec <= cols) {
        // a whole warp: lane 0 has the end of its first piece, lane 31 the start of the one behind its last: a piece in all,
        // of which a lane each stores a column
        if (off == 0) return;
        const bool head = lane < kPiece - off;
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t y = __shfl_sync(0xffffffffu, kHalf || lane == 0 ? u[k] : u[N - 4 + k], head ? 0 : 31);
            if ((kHalf ? lane >> 1 : lane) == k) x = y;
        }
        T *at = row + (head ? 0 : 31 * kVec + kVec - kPiece) - lane * kVec + lane;
        if (lane >= kPiece) return;
        if constexpr (kHalf)
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)(lane & 1 ? x >> 16 : x);
        else
            *reinterpret_cast<uint32_t *>(at) = x;
        return;
    }
    const bool next = off == 0 || (lane < 31 && col + 2 * kVec - off <= cols), rest = col - off + kVec <= cols;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        if (col + j >= cols || (j < kPiece - off ? mine : j < kVec - off ? rest : next)) continue;
        if constexpr (kHalf)
            reinterpret_cast<uint16_t *>(row)[j] = (uint16_t)(u[j >> 1] >> (16 * (j & 1)));
        else
            reinterpret_cast<uint32_t *>(row)[j] = u[j];
    }
}

// Eight fp32 values of a thread that wrote them itself, in two planes of four, so that a warp's accesses of 16 bytes lie
// side by side (32 bytes apart they meet in the same banks two by two).
__device__ __forceinline__ void write_planes(float *base, int vec, int vecs, const V8 &a) {
    float v[kVec];
    floats_of(a, v);
    reinterpret_cast<float4 *>(base)[vec] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(base)[vecs + vec] = make_float4(v[4], v[5], v[6], v[7]);
}
// Where column c of 8 * vecs stands in planes.
__device__ __forceinline__ int plane_of(int c, int vecs) { return (c & 4) * vecs + (c >> 3) * 4 + (c & 3); }
__device__ __forceinline__ V8 read_planes(const float *base, int vec, int vecs) {
    const uint4 *q = reinterpret_cast<const uint4 *>(base);
    return f32_pairs(q[vec], q[vecs + vec]);
}

// A thread's i-th eight columns. Only the last ones may be cut off by the row's end, or not there at all.
template <int MODE, int VPT>
struct Columns {
    int t, T, cols;
    bool has_last, cut;
    uint32_t last_lanes;  // that have the last ones
    __device__ __forceinline__ Columns(int t, int T, int cols) : t(t), T(T), cols(cols) {
        const int vec = t + (VPT - 1) * T, left = (cols + kVec - 1) / kVec - (vec - (t & 31));
        has_last = MODE == kAnyRow || vec * kVec < cols;
        cut = MODE == kAnyRow || (vec + 1) * kVec > cols;
        last_lanes = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
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
    // of a row that starts `shift` bytes into the pieces at `row` (where rows start anywhere)
    template <bool BF16>
    __device__ __forceinline__ V8 read(const char *row, int shift, int i) const {
        if (MODE == kAnyRow) return singles(i, [&](int c) { return read_one<BF16>(row + shift, c); });
        if (MODE == kShiftRow) return read_shifted<BF16>(row, shift, vec(i));
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
    // By the lanes for which none(i) is false.
    __device__ __forceinline__ void store(const RowMat &m, int64_t row, int i, const V8 &a) const {
        float v[kVec];
        floats_of(a, v);
        if (MODE == kAnyRow) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (i < VPT - 1 || col(i, j) < cols) store_one(m, row * m.ld + col(i, j), v[j]);
            return;
        }
        if (MODE != kShiftRow || m.fast) {
            store_row(m, row, vec(i) * kVec, cols, v);
            return;
        }
        const uint32_t lanes = i == VPT - 1 ? last_lanes : 0xffffffffu;
        if (m.bf16) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
            store_words(static_cast<__nv_bfloat16 *>(m.p) + row * m.ld, vec(i), cols, lanes, u);
        } else {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(v[k]);
            store_words(static_cast<float *>(m.p) + row * m.ld, vec(i), cols, lanes, u);
        }
    }
};

// The bytes that a row's copy starts before the row.
template <int MODE>
__device__ __forceinline__ int row_shift(const char *row) { return starts_anywhere(MODE) ? (int)(reinterpret_cast<uintptr_t>(row) & 15u) : 0; }
// The bytes of the whole 16-byte pieces of memory that hold a row.
__device__ __forceinline__ uint32_t window(const char *row, int bytes) { return (uint32_t)(((int)(reinterpret_cast<uintptr_t>(row) & 15u) + bytes + 15) & ~15); }

}  // namespace rlk
