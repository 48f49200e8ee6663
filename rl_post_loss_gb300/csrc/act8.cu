// Activations packed into 8 bits and read back (the format: act8.cuh).
//
// A thread takes 16 columns, half a block, so that a code store is 16 bytes and what is done once a part is spread
// over 16 columns: with 8 columns a thread the instructions bound packing (65536 x 6144 bf16: 238 us, against 211).
// A row's whole blocks are numbered in parts, so that two neighbouring lanes always hold one block; the threads of
// the grid step through all rows' parts together.
#include "act8.cuh"

namespace rlk {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 8;
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
        uint32_t a = max(act8_amax(v[0]), act8_amax(v[1]));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        if (!live) continue;
        const uint32_t b = act8_scale(a, p.a.e4m3);
        const uint2 lo = act8_encode(v[0], b, p.a.e4m3), hi = act8_encode(v[1], b, p.a.e4m3);
        uint8_t *codes = p.a.codes + at.row * p.a.ld_codes;
        if (col + kPart <= p.cols) {
            *reinterpret_cast<uint4 *>(codes + col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            store_codes(codes, col, p.cols, false, lo);
            store_codes(codes, col + kVec, p.cols, false, hi);
        }
        if ((at.part & 1) == 0) p.a.scales[at.row * p.a.ld_scales + (at.part >> 1)] = (uint8_t)b;
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

// Rows that start anywhere. Packing, a thread reads 8 columns one by one (the lines that a warp touches stay in L1);
// reading back, a warp takes eight blocks of a row and a lane one column of each, so that single stores lie side by
// side. 8191 x 2050 fp32 to e4m3: 20 us (a lane a column: 27); back: 25 us (8 columns a thread: 58).
struct AnyPlace {
    int64_t row, step_rows;
    int part, parts, step_parts;
    __device__ AnyPlace(int parts, int64_t i, int64_t all) : parts(parts) {
        row = i / parts;
        part = (int)(i - row * parts);
        step_rows = all / parts;
        step_parts = (int)(all - step_rows * parts);
    }
    __device__ void step() {
        row += step_rows;
        part += step_parts;
        if (part >= parts) {
            part -= parts;
            ++row;
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_pack_any_kernel(Act8Params p) {
    for (AnyPlace at(p.row_parts, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);; at.step()) {
        if (!__any_sync(0xffffffffu, at.row < p.rows)) break;
        const int col = at.part * kVec;
        const bool live = at.row < p.rows && col < p.cols;
        float v[kVec] = {};
        if (live) {
            const T *x = static_cast<const T *>(p.x.p) + at.row * p.x.ld + col;
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (col + j < p.cols) v[j] = (float)x[j];
        }
        const uint32_t b = act8_scale(act8_block_max(act8_amax(v)), p.a.e4m3);
        if (!live) continue;
        store_codes(p.a.codes + at.row * p.a.ld_codes, col, p.cols, p.a.fast, act8_encode(v, b, p.a.e4m3));
        if ((at.part & 3) == 0) p.a.scales[at.row * p.a.ld_scales + (at.part >> 2)] = (uint8_t)b;
    }
}

constexpr int kWide = 8 * kAct8Block;

__global__ void __launch_bounds__(kThreads) act8_unpack_any_kernel(Act8Params p) {
    const float most = p.x.bf16 ? __uint_as_float(0x7f7f0000u) : __uint_as_float(0x7f7fffffu);
    const int lane = threadIdx.x & 31;
    for (AnyPlace at(p.row_parts, (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), (int64_t)gridDim.x * (kThreads / 32)); at.row < p.rows; at.step()) {
        const uint8_t *codes = p.a.codes + at.row * p.a.ld_codes, *scales = p.a.scales + at.row * p.a.ld_scales + at.part * 8;
        const int col = at.part * kWide + lane;
        uint32_t c[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = at.part * kWide + j * kAct8Block < p.cols;
            b[j] = in ? scales[j] : 0u;
            c[j] = col + j * kAct8Block < p.cols ? codes[col + j * kAct8Block] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (col + j * kAct8Block >= p.cols) continue;
            const float v = act8_value(c[j], b[j], p.a.e4m3, most);
            if (p.x.bf16)
                (static_cast<__nv_bfloat16 *>(p.x.p) + at.row * p.x.ld)[col + j * kAct8Block] = __float2bfloat16_rn(v);
            else
                (static_cast<float *>(p.x.p) + at.row * p.x.ld)[col + j * kAct8Block] = v;
        }
    }
}

int grid_of(Act8Params &p) {
    p.row_parts = (p.cols + kAct8Block - 1) / kAct8Block * (kAct8Block / kPart);
    const int64_t blocks = (p.rows * p.row_parts + kThreads - 1) / kThreads;
    const int grid = (int)(blocks < kBlocks ? blocks : kBlocks);
    const int64_t all = (int64_t)grid * kThreads;
    p.step_rows = all / p.row_parts;
    p.step_parts = (int32_t)(all % p.row_parts);
    return grid;
}

// `lanes` threads a part.
int any_grid(Act8Params &p, int parts, int lanes) {
    p.row_parts = parts;
    const int64_t blocks = (p.rows * parts * lanes + kThreads - 1) / kThreads;
    return (int)(blocks < kBlocks ? blocks : kBlocks);
}

}  // namespace

cudaError_t launch_act8_pack(Act8Params p, cudaStream_t stream) {
    if (!p.x.fast || !p.a.fast) {
        const int grid = any_grid(p, (p.cols + kAct8Block - 1) / kAct8Block * (kAct8Block / kVec), 1);
        if (p.x.bf16)
            act8_pack_any_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
        else
            act8_pack_any_kernel<float><<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int grid = grid_of(p);
    if (p.x.bf16)
        act8_pack_kernel<__nv_bfloat16, Raw16><<<grid, kThreads, 0, stream>>>(p);
    else
        act8_pack_kernel<float, Raw32><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(Act8Params p, cudaStream_t stream) {
    if (!p.x.fast || !p.a.fast) {
        const int grid = any_grid(p, (p.cols + kWide - 1) / kWide, 32);
        act8_unpack_any_kernel<<<grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int grid = grid_of(p);
    act8_unpack_kernel<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace rlk
