// Activations packed into 8 bits and read back (the format: act8.cuh).
//
// A thread takes 16 columns, half a block, so that a code store is 16 bytes and what is done once a part is spread
// over 16 columns: with 8 columns a thread the instructions bound packing (65536 x 6144 bf16: 238 us, against 211 then).
// 65536 x 6144 bf16 to int8 takes 177 us (101% of the measured copy rate), back 193 us (93%), bound by memory.
// A row's whole blocks are numbered in parts, so that two neighbouring lanes always hold one block; the threads of
// the grid step through all rows' parts together.
#include "act8.cuh"

namespace rlk {

namespace {

constexpr int kThreads = 256;
// Five (reading back) or six blocks run on an SM at once: with 30 an SM all of them have the same number of turns, and a block
// that ends is followed by another. (65536 x 6144 bf16, there and back: 8 an SM 211 and 206 us, 5 188 and 191, 6 180 and 246, 30
// 177 and 193.)
constexpr int kBlocks = 152 * 30;
constexpr int kPart = 2 * kVec;

struct Place {
    int64_t row;
    int part;
    __device__ Place(const Act8Params &p) {
        const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        row = i / p.row_parts;
        part = (int)(i - row * p.row_parts);
    }
    __device__ void step(const Act8Params &p) {
        row += p.step_rows;
        part += p.step_parts;
        if (part >= p.row_parts) {
            part -= p.row_parts;
            ++row;
        }
    }
};

__device__ __forceinline__ void load_part(Raw16 (&r)[2], const __nv_bfloat16 *row, int col, int cols, int fast) {
    if (fast == 2 && col + kPart <= cols) {
        ld32(row + col, r[0].a, r[1].a);
        return;
    }
    load_raw(r[0], row, col, cols);
    if (col + kVec < cols) load_raw(r[1], row, col + kVec, cols);
}
__device__ __forceinline__ void load_part(Raw32 (&r)[2], const float *row, int col, int cols, int fast) {
    if (fast == 2 && col + kPart <= cols) {
        ld32(row + col, r[0].a, r[0].b);
        ld32(row + col + kVec, r[1].a, r[1].b);
        return;
    }
    load_raw(r[0], row, col, cols);
    if (col + kVec < cols) load_raw(r[1], row, col + kVec, cols);
}

// By all lanes of a warp, of which two neighbours hold a block.
__device__ __forceinline__ void pack_part(const Act8Params &p, int64_t row, int part, bool live, const float (&v)[2][kVec]) {
    uint32_t a = max(act8_amax(v[0]), act8_amax(v[1]));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    if (!live) return;
    const uint32_t b = act8_scale(a, p.a.e4m3);
    const uint2 lo = act8_encode(v[0], b, p.a.e4m3), hi = act8_encode(v[1], b, p.a.e4m3);
    uint8_t *codes = p.a.codes + row * p.a.ld_codes;
    const int col = part * kPart;
    if (p.a.fast && col + kPart <= p.cols) {
        *reinterpret_cast<uint4 *>(codes + col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
        store_codes(codes, col, p.cols, false, lo);
        store_codes(codes, col + kVec, p.cols, false, hi);
    }
    if ((part & 1) == 0) p.a.scales[row * p.a.ld_scales + (part >> 1)] = (uint8_t)b;
}

template <typename T, typename Raw>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(Act8Params p) {
    for (Place at(p);; at.step(p)) {
        if (!__any_sync(0xffffffffu, at.row < p.rows)) break;
        const int col = at.part * kPart;
        const bool live = at.row < p.rows && col < p.cols;
        float v[2][kVec] = {};
        if (live) {
            Raw r[2] = {};
            load_part(r, static_cast<const T *>(p.x.p) + at.row * p.x.ld, col, p.cols, p.x.fast);
            to_float(r[0], v[0]);
            to_float(r[1], v[1]);
            if (col + kPart > p.cols) {
                clip_row(v[0], col, p.cols);
                clip_row(v[1], col + kVec, p.cols);
            }
        }
        pack_part(p, at.row, at.part, live, v);
    }
}

__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(Act8Params p) {
    const float most = p.x.bf16 ? __uint_as_float(0x7f7f0000u) : __uint_as_float(0x7f7fffffu);
    for (Place at(p); at.row < p.rows; at.step(p)) {
        const int col = at.part * kPart;
        if (col >= p.cols) continue;
        const uint8_t *codes = p.a.codes + at.row * p.a.ld_codes;
        const uint4 c = ld16(codes + col);
        const uint32_t b = p.a.scales[at.row * p.a.ld_scales + (at.part >> 1)];
        const V8 lo = act8_decode(make_uint2(c.x, c.y), b, p.a.e4m3, most), hi = act8_decode(make_uint2(c.z, c.w), b, p.a.e4m3, most);
        float v[kVec], u[kVec];
        floats_of(lo, v);
        floats_of(hi, u);
        if (p.x.bf16 && p.x.fast == 2 && col + kPart <= p.cols) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
                w[4 + k] = pack_bf16x2(u[2 * k], u[2 * k + 1]);
            }
            st32(static_cast<__nv_bfloat16 *>(p.x.p) + at.row * p.x.ld + col, w);
        } else {
            store_row(p.x, at.row, col, p.cols, v);
            if (col + kVec < p.cols) store_row(p.x, at.row, col + kVec, p.cols, u);
        }
    }
}

// Rows that start anywhere come in the 16-byte pieces of memory that hold them: a thread loads the pieces that its 16
// columns lie in and shifts them into place, by whole words first. (8191 x 2050 fp32 to e4m3: 16 us; 8 columns a thread read
// one by one: 20.)
__device__ __forceinline__ void shift_words(uint32_t *w, int count, bool on, int by) {
#pragma unroll
    for (int i = 0; i < 20; ++i)
        if (i < count) w[i] = on ? w[i + by] : w[i];
}
template <int PIECES>
__device__ __forceinline__ void load_pieces(uint32_t (&w)[20], const void *first, int bytes) {  // of `bytes` from `first` on
    const char *q = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(first) & ~(uintptr_t)15);
    const char *end = static_cast<const char *>(first) + bytes;
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u);
        if (q + 16 * k < end) a = *reinterpret_cast<const uint4 *>(q + 16 * k);
        w[4 * k] = a.x, w[4 * k + 1] = a.y, w[4 * k + 2] = a.z, w[4 * k + 3] = a.w;
    }
}
__device__ __forceinline__ void load_any(float (&v)[2][kVec], const float *p, int count) {
    uint32_t w[20];
    load_pieces<5>(w, p, count * 4);
    const int shift = (int)(reinterpret_cast<uintptr_t>(p) >> 2) & 3;
    shift_words(w, 18, shift & 2, 2);
    shift_words(w, 16, shift & 1, 1);
#pragma unroll
    for (int j = 0; j < kPart; ++j) v[j / kVec][j % kVec] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void load_any(float (&v)[2][kVec], const __nv_bfloat16 *p, int count) {
    uint32_t w[20];
    load_pieces<3>(w, p, count * 2);
    const int shift = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 7;
    shift_words(w, 10, shift & 4, 2);
    shift_words(w, 9, shift & 2, 1);
#pragma unroll
    for (int j = 0; j < kPart / 2; ++j) {
        const uint32_t pair = __funnelshift_r(w[j], w[j + 1], (shift & 1) * 16);
        v[j / 4][2 * j % kVec] = bf16_lo(pair);
        v[j / 4][2 * j % kVec + 1] = bf16_hi(pair);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_pack_any_kernel(Act8Params p) {
    for (Place at(p);; at.step(p)) {
        if (!__any_sync(0xffffffffu, at.row < p.rows)) break;
        const int col = at.part * kPart;
        const bool live = at.row < p.rows && col < p.cols;
        float v[2][kVec] = {};
        if (live) {
            load_any(v, static_cast<const T *>(p.x.p) + at.row * p.x.ld + col, min(kPart, p.cols - col));
            if (col + kPart > p.cols) {
                clip_row(v[0], col, p.cols);
                clip_row(v[1], col + kVec, p.cols);
            }
        }
        pack_part(p, at.row, at.part, live, v);
    }
}

// Read back into rows that start anywhere, a thread takes the eight columns of a 32-byte (bf16: 16-byte) piece of memory, whose
// codes it shifts into place. (The same rows back: 18 us; single stores side by side, a lane a column: 25; eight columns a
// thread, stored one by one: 58.)
__global__ void __launch_bounds__(kThreads) act8_unpack_any_kernel(Act8Params p) {
    const float most = p.x.bf16 ? __uint_as_float(0x7f7f0000u) : __uint_as_float(0x7f7fffffu);
    const int es = p.x.bf16 ? 2 : 4;
    for (Place at(p); at.row < p.rows; at.step(p)) {
        char *x = static_cast<char *>(p.x.p) + at.row * p.x.ld * es;
        const int col = at.part * kVec - ((int)(reinterpret_cast<uintptr_t>(x) / es) & (kVec - 1)), lo = max(col, 0), hi = min(col + kVec, p.cols);
        if (lo >= hi) continue;
        const uint8_t *codes = p.a.codes + at.row * p.a.ld_codes, *scales = p.a.scales + at.row * p.a.ld_scales;
        const uint32_t b0 = scales[lo / kAct8Block], b1 = scales[(hi - 1) / kAct8Block];
        const int by = (int)(reinterpret_cast<uintptr_t>(codes) + col) & 3;
        uint32_t w[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int from = col - by + 4 * k;  // words that hold one of the codes at least
            w[k] = from + 4 > lo && from < hi ? *reinterpret_cast<const uint32_t *>(codes + from) : 0u;
        }
        const uint2 c = make_uint2(__funnelshift_r(w[0], w[1], by * 8), __funnelshift_r(w[1], w[2], by * 8));
        float v[kVec];
        floats_of(act8_decode(c, b0, p.a.e4m3, most), v);
        if (b0 != b1) {
            float u[kVec];
            floats_of(act8_decode(c, b1, p.a.e4m3, most), u);
            const int next = (lo / kAct8Block + 1) * kAct8Block;
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (col + j >= next) v[j] = u[j];
        }
        if (lo == col && hi == col + kVec) {
            if (p.x.bf16)
                store_vec(reinterpret_cast<__nv_bfloat16 *>(x), col, hi, true, v);
            else
                store_vec32(reinterpret_cast<float *>(x), col, v);
            continue;
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (col + j < lo || col + j >= hi) continue;
            if (p.x.bf16)
                reinterpret_cast<__nv_bfloat16 *>(x)[col + j] = __float2bfloat16_rn(v[j]);
            else
                reinterpret_cast<float *>(x)[col + j] = v[j];
        }
    }
}

// `parts` of a row, a thread each.
int grid_of(Act8Params &p, int parts) {
    p.row_parts = parts;
    const int64_t blocks = (p.rows * p.row_parts + kThreads - 1) / kThreads;
    const int grid = (int)(blocks < kBlocks ? blocks : kBlocks);
    const int64_t all = (int64_t)grid * kThreads;
    p.step_rows = all / p.row_parts;
    p.step_parts = (int32_t)(all % p.row_parts);
    return grid;
}
// Whole blocks in halves.
int halves(int cols) { return (cols + kAct8Block - 1) / kAct8Block * (kAct8Block / kPart); }

}  // namespace

cudaError_t launch_act8_pack(Act8Params p, cudaStream_t stream) {
    const int grid = grid_of(p, halves(p.cols));
    if (p.x.fast && p.a.fast) {
        if (p.x.bf16)
            act8_pack_kernel<__nv_bfloat16, Raw16><<<grid, kThreads, 0, stream>>>(p);
        else
            act8_pack_kernel<float, Raw32><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (p.x.bf16)
            act8_pack_any_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
        else
            act8_pack_any_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(Act8Params p, cudaStream_t stream) {
    if (p.x.fast && p.a.fast) {
        const int grid = grid_of(p, halves(p.cols));
        act8_unpack_kernel<<<grid, kThreads, 0, stream>>>(p);
    } else {
        const int grid = grid_of(p, (p.cols + 2 * kVec - 2) / kVec);
        act8_unpack_any_kernel<<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace rlk
